"""CPU check of a descriptor's tensors: codes and scales on one device."""
import pytest
import torch


@pytest.mark.parametrize("two_d", [False, True])
def test_codes_and_scales_are_on_one_device(two_d):
    import nvfp4_bit_microscaled_amd as m
    new = lambda n, device: torch.zeros(n, dtype=torch.uint8, device=device)  # noqa: E731
    nc, ns = m.fp8_tensor_bytes(40, 300, two_d)
    m.Fp8Tensor.wrap(new(nc, "cpu"), new(ns, "cpu"), 40, 300, two_d)
    for devices in (("cpu", "meta"), ("meta", "cpu")):
        with pytest.raises(ValueError, match="codes on"):
            m.Fp8Tensor.wrap(new(nc, devices[0]), new(ns, devices[1]), 40, 300, two_d)


def test_the_adapters_calls_keep_the_places_of_their_arguments():
    """A stream given by position stays the stream."""
    import inspect

    import nvfp4_bit_microscaled_amd as m
    for call, at in ((m.fp8_lora_fprop, 8), (m.fp8_lora_backward, 11)):
        assert list(inspect.signature(call).parameters)[at] == "stream"

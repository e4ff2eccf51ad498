"""Operands that are written and whose rows share bytes are refused on the host; no
GPU needed."""
import pytest
import torch

from mixed_precision_dense_tiled_amd import serving
from test_serving_binding import ALIASING, GB, NO_DEVICE, P, c_attn, kv, seqs

gpu_present = torch.cuda.is_available()


@pytest.mark.parametrize("change", [dict(ot=0), dict(oh=0), dict(ot=504), dict(oh=56), dict(ot=64, oh=64),
                                    dict(ot=64, oh=312), dict(ot=8, oh=512)])
def test_outputs_that_overlap_themselves(change):
    assert c_attn(**change) == ALIASING, change


def test_outputs_that_do_not():
    if gpu_present:
        pytest.skip("valid calls would run")
    for change in (dict(), dict(ot=520, oh=64), dict(ot=1024, oh=128), dict(ot=64, oh=320), dict(ot=72, oh=360)):
        assert c_attn(**change) == NO_DEVICE, change
    # one token, one head: its strides say nothing
    assert c_attn(sq=seqs(tokens=1), ot=0) == NO_DEVICE
    assert c_attn(kv(kv_heads=1), heads=1, oh=0, lt=1, ot=64) == NO_DEVICE


def test_caches_that_overlap_themselves():
    def append(**k):
        return serving._lib().paged_kv_append(kv(**k), seqs(), 0, P + 5 * GB, 128, 64, P + 6 * GB, 128, 64, None)

    for k in (dict(page_stride=0), dict(slot_stride=0), dict(head_stride=0), dict(page_stride=2040),
              dict(slot_stride=120), dict(head_stride=56), dict(slot_stride=64, head_stride=64)):
        assert append(**k) == ALIASING, k
    if not gpu_present:
        for k in (dict(), dict(slot_stride=64, head_stride=1024), dict(page_stride=64, slot_stride=640, head_stride=10240),
                  dict(page_stride=4096, slot_stride=256, head_stride=72), dict(pages=1, page_stride=0),
                  dict(kv_heads=1, head_stride=0)):
            assert append(**k) == NO_DEVICE, k
        # reading it is fine: one page for all, one head for all
        assert c_attn(kv(page_stride=0)) == NO_DEVICE and c_attn(kv(head_stride=0)) == NO_DEVICE

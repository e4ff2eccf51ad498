"""Sizes that a launch cannot hold are refused on the host; no GPU needed."""
import torch

from mixed_precision_dense_tiled_amd import serving
from test_serving_binding import INVALID, NO_DEVICE, P, kv, seqs

gpu_present = torch.cuda.is_available()
FAR = 1 << 44          # bytes between operands that are large here
# a launch holds fewer than 2^32 threads along x
GROUPS = (2 ** 32 - 1) // 256


def lib():
    return serving._lib()


def test_rows_of_logits():
    def forward(rows, vocab):
        return lib().token_logprobs(0, rows, vocab, P, vocab, P + FAR, 0, P + 2 * FAR, P + 3 * FAR, P + 4 * FAR, None,
                                    None, None, 0, None)

    def backward(rows, vocab):
        return lib().token_logprobs_backward(0, rows, vocab, P, vocab, P + FAR, P + 2 * FAR, P + 3 * FAR, P + 4 * FAR,
                                             None, P + 5 * FAR, vocab, None)

    for call in (forward, backward):
        assert call(GROUPS + 1, 2) == INVALID and call(1 << 30, 2) == INVALID
        if not gpu_present:
            assert call(GROUPS, 2) == NO_DEVICE
    # two workgroups a row in the gradient's launch, one in the other
    assert backward(GROUPS // 2 + 1, 10000) == INVALID
    if not gpu_present:
        assert forward(GROUPS // 2 + 1, 10000) == NO_DEVICE


def test_new_tokens():
    def append(tokens):
        return lib().paged_kv_append(kv(dim=16, head_stride=16, slot_stride=32, page_stride=512), seqs(tokens=tokens), 0,
                                     P + FAR, 32, 16, P + 2 * FAR, 32, 16, None)

    assert append(GROUPS * 8 + 1) == INVALID and append(1 << 30) == INVALID
    if not gpu_present:
        assert append(GROUPS * 8) == NO_DEVICE


def test_single_tokens_in_one_launch():
    """Short caches take a workgroup of 512 threads to 16 rows of a sequence, where
    a launch holds them; more are shared out over a fixed number of workgroups."""
    most = (2 ** 32 - 1) // 512

    def workspace(n):
        s = seqs(seqs=n, tokens=n, width=1, ld_table=1, table=P + FAR, cu_q=P + 2 * FAR, lens=P + 3 * FAR)
        return lib().paged_attention_workspace(kv(kv_heads=1, dim=16, head_stride=16, slot_stride=16, page_stride=256),
                                               s, 1)

    n = most - most // 17       # n + n / 16 tiles
    assert n + n // 16 <= most < (n + 20) + (n + 20) // 16
    assert workspace(n) == 0 and workspace(n + 20) > 0 and workspace(1 << 28) > 0


def test_rows_of_a_page_table():
    def view(rows):
        return serving._Pages(P, 1 << 20, 4096, 4096, 2, 8, 16, P + FAR, P + 2 * FAR, 1, P + 3 * FAR, rows, 1)

    def fork(rows):
        return lib().cache_fork(view(rows), P + 4 * FAR, None, P + 5 * FAR, lib().cache_pages_workspace(8, rows), None)

    def free(rows):
        return lib().cache_free(view(rows), P + 4 * FAR, None)

    for call in (fork, free):
        assert call(GROUPS + 1) == INVALID and call(1 << 30) == INVALID
        if not gpu_present:
            assert call(GROUPS) == NO_DEVICE

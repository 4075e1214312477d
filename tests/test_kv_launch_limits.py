"""Key/value cache calls whose launch would have 2^32 threads in a row or more, which the runtime counts in 32 bits and drops
the rest of: attention, append and read refuse them before any launch, page management runs them."""
import ctypes

import pytest
import torch

import nvfp4_block_scaled_amd as nv

FAKE = 0x10000            # never dereferenced
B = ctypes.byref


def cache(heads=16):
    return nv._Cache(FAKE, 8, heads * 16 * 16 * 9 // 8, 16, heads, 16, 0, None, None)


def rows(heads=16):
    return nv._Rows(FAKE, 16 * heads, 16)


def attention(batch, heads):
    """One token for each sequence; a workgroup for each and KV head. Without a workspace, a call that is taken says so."""
    return nv.lib().nvfp4_kv_attention(B(cache(heads)), rows(heads), 1, batch, heads, FAKE, 100, 100, FAKE, None, batch, 1,
                                       B(nv._Mask(0.1, 1, 0, None, 0)), rows(heads), None, None, 0, None)


def test_attention():
    assert attention(1 << 20, 16) == nv.ERR_SHAPE and attention(1 << 19, 48) == nv.ERR_SHAPE
    assert attention((1 << 20) - 1000, 15) == nv.ERR_WORKSPACE
    need = nv.lib().nvfp4_kv_attention_workspace_bytes
    assert need(B(cache()), 1 << 20, 16, 1 << 20, 100, 1) == 0 and need(B(cache(15)), 1 << 20, 15, 1 << 20, 100, 1) > 0


def test_append_and_read():
    tokens = 1 << 33
    assert nv.lib().nvfp4_kv_append(B(cache()), rows(), rows(), nv._Rows(None, 0, 0), nv._Rows(None, 0, 0), 1, tokens, 0, FAKE, None, None) \
        == nv.ERR_SHAPE
    assert nv.lib().nvfp4_kv_read(B(cache()), FAKE, 1 << 28, 1, rows(), rows(), None) == nv.ERR_SHAPE


B24 = 1 << 24             # sequences, at the limit of the tables


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
def test_resize_of_many_sequences():
    """All empty but the last two: one gives back its pages 5 and 6, and the other takes them. Rows carry over to another table."""
    table = torch.arange(2 * B24, dtype=torch.int32, device="cuda").remainder_(7).view(B24, 2)
    lens, new = torch.zeros(B24, dtype=torch.int32, device="cuda"), torch.zeros(B24, dtype=torch.int32, device="cuda")
    table[-1] = ints(5, 6)
    table[-2] = -1
    lens[-1], new[-2] = 20, 17
    refs = ints(1, 1, 1, 1, 1, 1, 1, 0)
    want = table.clone()
    want[-1], want[-2] = -1, ints(5, 6)
    out, counts, short = nv.nvfp4_kv_resize(table, lens, new, refs, 16, out_table=torch.full_like(table, 99))
    assert torch.equal(out, want) and counts.tolist() == [1, 1, 1, 1, 1, 1, 1, 0] and int(short) == 0


@pytest.mark.gpu
def test_fork_into_many_children():
    """All of no parent but the first and the last."""
    pages = torch.arange(8 * 48, dtype=torch.int32, device="cuda").to(torch.uint8).view(8, 48)
    parents = torch.full((B24,), -1, dtype=torch.int32, device="cuda")
    parents[0] = parents[-1] = 0
    refs = ints(1, 1, 0, 0, 0, 0, 0, 0)
    kept = pages[1].clone()
    out, counts, short = nv.nvfp4_kv_fork(pages, ints(0, 1)[None], ints(20), refs, parents, 16,
                                          out_table=torch.full((B24, 2), 99, dtype=torch.int32, device="cuda"))
    assert out[0].tolist() == [0, 2] and out[-1].tolist() == [0, 3] and bool((out[1:-1] == -1).all())
    assert counts.tolist() == [3, 1, 1, 1, 0, 0, 0, 0] and int(short) == B24 - 2
    assert torch.equal(pages[2], kept) and torch.equal(pages[3], kept)

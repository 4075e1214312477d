"""Tokens to experts and back where the sorted rows pass the memory-side cache, sorts and rows on two streams at once, and all
of it captured. Values are small integers, so every result is exact: gradients' dots of 4003 products of at most 8 stay below
2^24, sums of eight rows with weights of 1/2, 1 and 2 below 2^8 in halves, which BF16 holds."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_amd as nv
from oracle import moe

pytestmark = pytest.mark.gpu


def integers(g, lo, hi, shape, dtype):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(dtype)


def choices(g, T, top, experts):
    return torch.rand((T, experts), generator=g, device="cuda").argsort(1)[:, :top]


@pytest.mark.parametrize("T,top,width,dtype,pad", [(4200, 8, 4003, torch.bfloat16, 5), (9000, 4, 3800, torch.float16, 0),
                                                   (8400, 8, 1001, torch.float32, 0)])
def test_rows_past_the_cache(T, top, width, dtype, pad):
    """Over 256 MB of sorted rows, of an odd width, in a wider matrix; one choice in four takes no part."""
    g = torch.Generator("cuda").manual_seed(T)
    ids = choices(g, T, top, 64)
    ids[torch.rand(ids.shape, generator=g, device="cuda") < 0.25] = -1
    offsets, tokens, places = nv.nvfp4_moe_sort(ids, 64)
    assert T * top * width * torch.empty(0, dtype=dtype).element_size() > 256 << 20
    used, place = int(offsets[-1]), places.long()
    x = integers(g, -2, 2, (T, width), dtype)
    room = torch.full((T * top, width + pad), 9.0, dtype=dtype, device="cuda")
    rows = nv.nvfp4_moe_gather(x, places, out=room[:, :width])
    assert torch.equal(rows[:used], x[tokens[:used].long()])
    assert bool((room[used:] == 9.0).all()) and bool((room[:, width:] == 9.0).all())

    weights = torch.exp2(integers(g, -1, 1, (T, top), torch.float32))
    y = integers(g, -4, 4, (T * top, width), dtype)
    want, plain = torch.zeros((T, width), device="cuda"), torch.zeros((T, width), device="cuda")
    for j in range(top):
        part = torch.where(place[:, j:j + 1] >= 0, y[place[:, j].clamp(min=0)].float(), 0.0)
        plain += part
        want += weights[:, j:j + 1] * part
    assert torch.equal(nv.nvfp4_moe_combine(y, places, weights), want.to(dtype))
    assert torch.equal(nv.nvfp4_moe_gather_backward(y, places), plain.to(dtype))

    grad = integers(g, -2, 2, (T, width), dtype)
    room.fill_(9.0)
    grad_y, grad_w = nv.nvfp4_moe_combine_backward(grad, y, places, weights, grad_y=room[:, :width])
    for j in range(top):
        at = place[:, j] >= 0
        assert torch.equal(grad_y[place[at, j]], (weights[at, j:j + 1] * grad[at]).to(dtype))
        dots = (grad.float() * y[place[:, j].clamp(min=0)].float()).sum(1)
        assert torch.equal(grad_w[:, j], torch.where(at, dots, 0.0))
    assert bool((room[used:] == 9.0).all()) and bool((room[:, width:] == 9.0).all())


@pytest.mark.parametrize("T,top,experts", [(1023, 4, 64), (4096, 1, 896), (4096, 1, 897), (4097, 1, 64), (40000, 8, 100), (1, 5000, 3)])
def test_sorts_around_the_passes(T, top, experts):
    """What one workgroup places in a pass and a pair more; chunks of two passes; one token with many choices."""
    ids = np.random.default_rng(T).integers(-1, experts + 1, (T, top)).astype(np.int32)
    for got, want in zip(nv.nvfp4_moe_sort(torch.from_numpy(ids).cuda(), experts), moe.sort(ids, experts)):
        np.testing.assert_array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("T,experts", [(40, 60), (5000, 300)])
def test_two_dispatches_at_once(T, experts):
    g = torch.Generator("cuda").manual_seed(T)
    ids = [choices(g, T, 4, experts).int() for _ in range(2)]
    x = [integers(g, -4, 4, (T, 136), torch.bfloat16) for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                o, t, p = nv.nvfp4_moe_sort(ids[i], experts)
                got[i].append((o, t, p, nv.nvfp4_moe_gather(x[i], p)))
    torch.cuda.synchronize()
    for i in range(2):
        want = moe.sort(ids[i].cpu().numpy(), experts)
        for o, t, p, rows in got[i]:
            for a, b in zip((o, t, p), want):
                np.testing.assert_array_equal(a.cpu().numpy(), b)
            assert torch.equal(rows, x[i][t.long()])


@pytest.mark.parametrize("T,experts,dtype", [(3, 8, torch.int64), (600, 64, torch.int32), (3000, 128, torch.int32)])
def test_the_way_there_and_back_captured(T, experts, dtype):
    """A graph of sort, gather, combine and the gradients, replayed on new choices between eager calls."""
    g = torch.Generator("cuda").manual_seed(T)
    top, width = 4, 200
    ids, x = torch.empty((T, top), dtype=dtype, device="cuda"), torch.empty((T, width), dtype=torch.bfloat16, device="cuda")
    weights = torch.exp2(integers(g, -1, 1, (T, top), torch.float32))

    def run(ids, x):
        o, t, p = nv.nvfp4_moe_sort(ids, experts)
        rows = nv.nvfp4_moe_gather(x, p)
        out = nv.nvfp4_moe_combine(rows, p, weights)
        return (o, t, p, rows, out, nv.nvfp4_moe_gather_backward(rows, p)) + nv.nvfp4_moe_combine_backward(x, rows, p, weights)
    news = [(choices(g, T, top, experts).to(dtype), integers(g, -4, 4, (T, width), torch.bfloat16)) for _ in range(3)]
    want = [[t.clone() for t in run(*n)] for n in news]
    side = torch.cuda.Stream()
    ids.copy_(news[0][0])
    x.copy_(news[0][1])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        run(ids, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(ids, x)
    for k in (0, 1, 2, 0):
        ids.copy_(news[k][0])
        x.copy_(news[k][1])
        graph.replay()
        run(*news[(k + 1) % 3])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[k]))

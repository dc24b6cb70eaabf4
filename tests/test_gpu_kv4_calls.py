"""Calls of the 4-bit cache that are rare but allowed, and refusals that must name their
reason."""

import ctypes

import numpy as np
import pytest
import torch

import block_causal_streaming_sa_b200 as sa
from oracle import kv4
from test_gpu_kv4 import BF, Pair, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("add_weight", [False, True])
def test_attend_without_query_tokens_as_the_first_call(add_weight):
    c = sa.QuantKVCache(2, 2, 64, 128)
    none = torch.empty((2, 0, 4, 64), dtype=BF, device="cuda")
    lse = torch.empty((2, 4, 0), device="cuda")
    out = c.attend(none, lse=lse, add_weight=add_weight)
    assert out.shape == none.shape and c._workspaces == []
    some = normal("none", (2, 3, 2, 64), BF).cuda()
    c.append(some, some)
    weight = c.weight.clone()
    c.attend(none, out=none, add_weight=add_weight, causal=True)
    assert torch.equal(c.weight.view(torch.uint8), weight.view(torch.uint8))
    assert c.check() == sa.SA_OK


def test_unsupported_sizes_are_refused_by_the_library_whatever_came_before():
    c = sa.QuantKVCache(1, 1, 96, 128)
    q = torch.zeros((1, 1, 1, 96), dtype=BF, device="cuda")
    for call in (lambda: c.attend(q), lambda: c.evict(5), lambda: c.append(q, q)):
        with pytest.raises(sa.SaError, match="head_dim must be 64 or 128") as e:
            call()
        assert e.value.status == sa.SA_ERR_UNSUPPORTED


def test_a_capture_on_the_stream_passed_in_needs_the_workspace_too():
    """The call's stream captures, the current one does not."""
    p = Pair(1, 1, 64, 128)
    p.append("caps", 10)
    q = normal("capsq", (1, 1, 1, 64), BF).cuda()
    out = torch.empty_like(q)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="before capturing"):
        with torch.cuda.graph(graph, stream=side):
            with torch.cuda.stream(other):
                p.gpu.attend(q, out=out, stream=side)
    torch.cuda.synchronize()
    assert p.gpu._workspaces == []
    want = p.gpu.attend(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        with torch.cuda.stream(other):
            p.gpu.attend(q, out=out, stream=side)
    graph.replay()
    assert torch.equal(out, want)


def test_a_launch_that_fails_ends_the_call_with_an_error():
    """On a stream whose capture has become invalid every launch is refused on the host: each
    call says so, and the cache works again once the capture has ended."""
    c = sa.QuantKVCache(1, 1, 64, 9088)
    K = normal("fail", (1, 90, 1, 64), BF).cuda()
    c.append(K, K)
    out, other = torch.empty_like(K), torch.empty_like(K)
    want = c.attend(K, add_weight=True)
    one = c.attend(K[:, :1], add_weight=True)
    seq, weight = c.seq.clone(), c.weight.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    driver, relaxed = ctypes.CDLL("libcuda.so.1"), 2
    stream, graph = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p()
    assert driver.cuStreamBeginCapture_v2(stream, relaxed) == 0
    try:
        assert c.check(stream=side) == sa.SA_ERR_CUDA  # waiting for it makes the capture invalid
        for call in (lambda: c.append(K, K, stream=side),
                     lambda: c.read(0, out, other, stream=side),
                     lambda: c.attend(K, out=out, add_weight=True, stream=side),
                     lambda: c.attend(K[:, :1], out=out[:, :1], add_weight=True, stream=side),
                     lambda: c.attend(K[:, :30], out=out[:, :30], add_weight=True, stream=side),
                     lambda: c.evict(20, stream=side), lambda: c.reset(stream=side)):
            with pytest.raises(sa.SaError) as e:
                call()
            assert e.value.status == sa.SA_ERR_CUDA and "kv4: " in sa.last_error()
    finally:
        assert driver.cuStreamEndCapture(stream, ctypes.byref(graph)) != 0
    torch.cuda.synchronize()
    assert torch.equal(c.seq, seq) and torch.equal(c.weight[:, :, :90], weight[:, :, :90])
    assert torch.equal(c.attend(K), want) and torch.equal(c.attend(K[:, :1]), one)
    c.append(K, K, stream=side)
    assert c.check(stream=side) == sa.SA_OK and c.seq[0].tolist() == [180]


@pytest.mark.parametrize("H,n,keep", [(40, 20_000, 15_001), (70, 9000, 8999), (148, 12_000, 7000),
                                      (150, 45_000, 30_000)])
def test_evict_many_heads_of_long_rows(H, n, keep):
    """Heads that share the device in clusters of every size, and rows whose keys do not fit one
    block's shared memory though every SM has a head."""
    c = sa.QuantKVCache(1, H, 64, -(-n // 128) * 128)
    g = torch.Generator(device="cuda").manual_seed(n)
    K = torch.randn((1, n, H, 64), generator=g, device="cuda").bfloat16()
    c.append(K, K)
    w = torch.randint(0, 5000, c.weight.shape, generator=g, device="cuda").float()
    c.weight.copy_(w)
    kc = c.k_codes.clone()
    c.evict(keep, first=7, recent=300)
    for h in (0, 1, H // 2, H - 1):
        src = torch.tensor(kv4.rows_after_eviction(w[0, h, :n].cpu().numpy(), np.arange(n), n,
                                                   keep, 7, 300), device="cuda")
        assert torch.equal(c.weight[0, h, :keep], w[0, h, src])
        assert torch.equal(c.k_codes[0, h, :keep], kc[0, h, src])
        assert torch.equal(c.pos[0, h, :keep], src.int())
    assert c.seq[0].tolist() == [keep]


@pytest.mark.parametrize("D", [64, 128])
def test_many_row_attention_between_library_matrix_products(D):
    """Attention of many rows, with weights, in a stream full of matrix products of another
    library, without a pause: the bits are those of calls that wait."""
    p = Pair(1, 4, D, 2048)
    p.append(("mix", D), 2000)
    Q = normal(("mixq", D), (1, 300, 8, D), BF).cuda()
    a = torch.randn((2048, 2048), device="cuda").bfloat16()
    p.gpu.weight.zero_()
    lse = torch.empty((1, 8, 300), device="cuda")
    want = p.gpu.attend(Q, lse=lse, add_weight=True)
    weight, prod = p.gpu.weight.clone(), a @ a
    torch.cuda.synchronize()
    for _ in range(20):
        p.gpu.weight.zero_()
        x = a @ a
        out = p.gpu.attend(Q, add_weight=True)
        y = a @ a
        again = p.gpu.attend(Q)
        assert torch.equal(out, want) and torch.equal(again, want)
        assert torch.equal(x, prod) and torch.equal(y, prod)
        assert torch.equal(p.gpu.weight[:, :, :2000], weight[:, :, :2000])
    assert p.gpu.check() == sa.SA_OK

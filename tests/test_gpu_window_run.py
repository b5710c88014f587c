"""The windowed and the 4-bit operators as they are used: a prompt, its cache in 4 bits,
steps over both kinds of cache and a later chunk of the prompt, against the fp64
reference; captured into a graph, from several threads, on a stream given to the call,
and in front of a programmatic dependent, to the bits of the same calls made alone.

Tolerances: those of the windowed prefill and decode tests (cache_common derives
them), and of the 4-bit ones.
"""

import json
import os
import subprocess
import sys
import threading

import numpy as np
import pytest

from causal_gqa_prefill_gb300 import (ATTN_ERR_UNSUPPORTED, ATTN_OK, attn_decode,
                                      attn_decode4, attn_decode4_workspace_bytes,
                                      attn_decode_window, attn_decode_window_workspace_bytes,
                                      attn_device_check, attn_pack4, attn_prefill_window,
                                      attn_prefill_window_backward,
                                      attn_prefill_window_bwd_workspace_bytes, attn_unpack4)
from causal_gqa_prefill_gb300 import workloads as W
from gpu_common import to_np
from oracle import cache4
from oracle import window as ow
from test_gpu_cache4 import check_step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from causal_gqa_prefill_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def normal(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def check_rows(o, lse, ref, d, rows=slice(None)):
    o_r, lse_r, o_abs, s_abs = ref
    bound = 2.0 ** -8 * ((1 + 2.0 ** -6) * o_abs + np.abs(o_r))
    assert (np.abs(to_np(o) - o_r) <= bound)[:, rows].all()
    bound = (d + 2) * 2.0 ** -24 * s_abs + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse_r)
    assert (np.abs(to_np(lse) - lse_r) <= bound)[:, :, rows].all()


def test_a_prompt_its_steps_and_a_later_chunk():
    B, C, n_q, n_kv, d, win, sinks = 2, 512, 8, 2, 128, 96, 4
    lens = [400, 250]                                    # a batch padded to 400 rows
    q, k, v = W.make_inputs(W.custom(B, 400, n_q, n_kv, d), "cuda", seed=60)
    for b in range(B):
        for x in (q, k, v):
            x[b, lens[b]:] = 0
    o, lse = attn_prefill_window(q, k, v, win, sinks)
    ref = ow.attention(to_np(q), to_np(k), to_np(v), win, sinks)
    for b in range(B):
        check_rows(o[b:b + 1], lse[b:b + 1], [x[b:b + 1] for x in ref], d, slice(lens[b]))

    # the cache in bf16 and in 4 bits: rows behind a sequence keep what they held
    kc, vc = (torch.full((B, C, n_kv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    k4, v4 = (torch.full((B, n_kv, C, 80), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    n = i32(*lens)
    for b in range(B):
        kc[b, :lens[b]], vc[b, :lens[b]] = k[b, :lens[b]], v[b, :lens[b]]
    attn_pack4(k, v, k4, v4, counts=n)
    for b in range(B):
        assert (k4[b, :, lens[b]:] == 255).all() and (v4[b, :, lens[b]:] == 255).all()

    rows = torch.arange(B, device="cuda")
    for step in range(6):
        q1, k1, v1 = (normal(70 + 3 * step + i, B, 1, h, d) for i, h in enumerate((n_q, n_kv, n_kv)))
        attn_pack4(k1, v1, k4, v4, n)
        kc[rows, n.long()], vc[rows, n.long()] = k1[:, 0], v1[:, 0]
        n += 1
        o, lse = attn_decode_window(q1, kc, vc, n, win, sinks)
        check_rows(o, lse, ow.decode_rows(to_np(q1), to_np(kc), to_np(vc), n.tolist(), win, sinks), d)
        o4, lse4 = attn_decode4(q1, k4, v4, n, window=win, sinks=sinks)
        check_step(q1, k4, v4, n.tolist(), o4, lse4, win, sinks)
    assert attn_device_check() == ATTN_OK

    # a later chunk of the first sequence's prompt, behind its rows read back
    have, more = int(n[0]), 70
    ku, vu = attn_unpack4(k4[:1], v4[:1], have)
    for got, c in ((ku, k4), (vu, v4)):
        want = cache4.rounded(c[:1, :, :have].cpu().numpy()).transpose(0, 2, 1, 3)
        assert np.array_equal(to_np(got), want)
    q2, k2, v2 = (normal(90 + i, 1, more, h, d) for i, h in enumerate((n_q, n_kv, n_kv)))
    K, V = torch.cat((ku, k2), 1), torch.cat((vu, v2), 1)
    o, lse = attn_prefill_window(q2, K, V, win, sinks)
    check_rows(o, lse, ow.attention(to_np(q2), to_np(K), to_np(V), win, sinks), d)
    attn_pack4(k2, v2, k4[:1], v4[:1], n[:1])
    n[0] += more
    o, lse = attn_decode4(q2[:, -1:].contiguous(), k4[:1], v4[:1], n[:1], window=win, sinks=sinks)
    check_step(q2[:, -1:], k4[:1], v4[:1], [have + more], o, lse, win, sinks)
    assert attn_device_check() == ATTN_OK


def inputs(seed, B=2, L=700, n_q=8, n_kv=2, d=128):
    x = {n: normal(seed + i, B, L, h, d)
         for i, (n, h) in enumerate((("q", n_q), ("k", n_kv), ("v", n_kv), ("do", n_q)))}
    x["qd"] = normal(seed + 4, B, 1, n_q, d)
    g = torch.Generator(device="cuda").manual_seed(seed + 5)
    x["lens"] = torch.randint(100, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    return x


def outputs(x):
    B, L, n_q, d = x["q"].shape
    n_kv = x["k"].shape[2]
    f32 = dict(dtype=torch.float32, device="cuda")
    u8 = dict(dtype=torch.uint8, device="cuda")
    sizes = dict(ws_bwd=attn_prefill_window_bwd_workspace_bytes(B, L, n_q, n_kv, d, 200, 3),
                 ws_win=attn_decode_window_workspace_bytes(B, L, n_q, n_kv, window=200, sinks=3),
                 ws_four=attn_decode4_workspace_bytes(B, L, n_q, n_kv))
    y = dict(o=torch.zeros_like(x["q"]), lse=torch.zeros(B, n_q, L, **f32),
             dq=torch.zeros_like(x["q"]), dk=torch.zeros_like(x["k"]), dv=torch.zeros_like(x["v"]),
             od=torch.zeros_like(x["qd"]), ld=torch.zeros(B, n_q, 1, **f32),
             k4=torch.full((B, n_kv, L, 80), 17, **u8), v4=torch.full((B, n_kv, L, 80), 17, **u8),
             o4=torch.zeros_like(x["qd"]), l4=torch.zeros(B, n_q, 1, **f32),
             ku=torch.zeros_like(x["k"]), vu=torch.zeros_like(x["v"]))
    y.update({n: torch.full((size,), 255, **u8) for n, size in sizes.items()})
    return y


def all_calls(x, y, stream=None):
    """Every call, into the outputs y; the forward's row results feed the backward."""
    s = dict(stream=stream)
    attn_prefill_window(x["q"], x["k"], x["v"], 200, 3, out=y["o"], lse=y["lse"], **s)
    attn_prefill_window_backward(x["q"], x["k"], x["v"], y["o"], y["lse"], x["do"], 200, 3,
                                 workspace=y["ws_bwd"], dq=y["dq"], dk=y["dk"], dv=y["dv"], **s)
    attn_decode_window(x["qd"], x["k"], x["v"], x["lens"], 200, 3, out=y["od"], lse=y["ld"],
                       workspace=y["ws_win"], **s)
    attn_pack4(x["k"], x["v"], y["k4"], y["v4"], counts=x["lens"], **s)
    attn_decode4(x["qd"], y["k4"], y["v4"], x["lens"], out=y["o4"], lse=y["l4"],
                 workspace=y["ws_four"], **s)
    attn_unpack4(y["k4"], y["v4"], y["ku"].shape[1], k=y["ku"], v=y["vu"], **s)


def results(y):
    return {n: t.clone() for n, t in y.items() if not n.startswith("ws")}


def same(a, b):
    # (rows of the cache that nothing was packed into unpack to whatever they held)
    return all(torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)) for n in b)


def test_captured_into_one_graph():
    x = inputs(200)
    y = outputs(x)
    all_calls(x, y)                                      # the one-time set-up of each family
    torch.cuda.synchronize()
    assert attn_device_check() == ATTN_OK
    eager = results(y)
    fresh = outputs(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        all_calls(x, y)
    for n, t in fresh.items():
        y[n].copy_(t)
    graph.replay()
    torch.cuda.synchronize()
    assert same(y, eager)
    for n, t in inputs(300).items():                     # new values, lengths among them
        x[n].copy_(t)
    y2 = outputs(x)
    all_calls(x, y2)
    for n, t in fresh.items():
        y[n].copy_(t)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert attn_device_check() == ATTN_OK
    assert same(y, results(y2)) and not same(y, eager)


def test_two_graphs_with_one_workspace():
    """Captured one behind the other with the same workspaces, replayed in both orders."""
    xs = [inputs(400), inputs(500, L=333)]
    ys = [outputs(x) for x in xs]
    for n in ("ws_bwd", "ws_win", "ws_four"):
        shared = max((y[n] for y in ys), key=lambda t: t.numel())
        for y in ys:
            y[n] = shared
    for x, y in zip(xs, ys):
        all_calls(x, y)
    want = [results(y) for y in ys]
    graphs = []
    for x, y in zip(xs, ys):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            all_calls(x, y)
    for order in ((0, 1, 0), (1, 0)):
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(same(y, w) for y, w in zip(ys, want)), order
    assert attn_device_check() == ATTN_OK


def test_on_a_stream_given_to_the_call():
    """The inputs are made, late, on the stream that the calls are given."""
    x = inputs(600)
    y = outputs(x)
    all_calls(x, y)
    want = results(y)
    side = torch.cuda.Stream()
    late = {n: torch.zeros_like(t) for n, t in x.items()}
    y = outputs(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        for n, t in x.items():
            late[n].copy_(t)
    all_calls(late, y, stream=side)
    side.synchronize()
    assert attn_device_check() == ATTN_OK
    assert same(y, want)


def test_threads_at_once():
    xs = [inputs(700 + 10 * i, L=300 + 97 * i) for i in range(4)]

    def calls(x):
        y = outputs(x)
        all_calls(x, y)
        o, lse = attn_prefill_window(x["q"], x["k"], x["v"], 64)
        more = dict(zip(("wq", "wk", "wv"), attn_prefill_window_backward(
            x["q"], x["k"], x["v"], o, lse, x["do"], 64)))
        more["wo"], more["wl"] = attn_decode4(x["qd"], y["k4"], y["v4"], x["lens"], window=50)
        return {**results(y), **more}

    alone = [calls(x) for x in xs]
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = [calls(xs[i]) for _ in range(10)]
                torch.cuda.current_stream().synchronize()
        except Exception as e:                                           # noqa: BLE001
            errors.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and attn_device_check() == ATTN_OK
    for i, want in enumerate(alone):
        assert all(same(run, want) for run in got[i]), i


@pytest.mark.parametrize("L,n_q,n_kv,win,sinks", [
    (1024, 16, 1, 900, 0),               # few key tiles: all of them in pieces
    (1024, 16, 1, 30, 200),              # the sinks' tiles in pieces
    (1024, 16, 8, 700, 0),
])
def test_programmatic_successor_sees_complete_gradients(L, n_q, n_kv, win, sinks):
    """A decode step, whose kernels are programmatic dependents, reads dK and dV as its
    cache straight after the backward."""
    q, k, v = W.make_inputs(W.custom(1, L, n_q, n_kv, 128), "cuda", seed=51)
    do, qd = normal(52, *q.shape), normal(53, 1, 1, n_q, 128)
    o, lse = attn_prefill_window(q, k, v, win, sinks)
    torch.cuda.synchronize()
    _, dk, dv = attn_prefill_window_backward(q, k, v, o, lse, do, win, sinks)
    first = attn_decode(qd, dk, dv)                      # no host sync in between
    torch.cuda.synchronize()
    assert attn_device_check() == ATTN_OK
    again = attn_decode(qd, dk, dv)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


_FIRST_CALL = r"""
import json, torch
import causal_gqa_prefill_gb300 as cg
torch.cuda.set_device(0)
q = torch.randn(1, 256, 4, 128, device="cuda").to(torch.bfloat16)
k = torch.randn(1, 256, 2, 128, device="cuda").to(torch.bfloat16)
v, qd, do = torch.randn_like(k), q[:, -1:].contiguous(), torch.randn_like(q)
k4 = torch.zeros(1, 2, 256, 80, dtype=torch.uint8, device="cuda")
v4 = torch.zeros_like(k4)
o, lse = torch.randn_like(q), torch.randn(1, 4, 256, device="cuda")
lens = torch.tensor([200], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
res = {}
def in_capture(name, fn):
    g = torch.cuda.CUDAGraph()
    try:
        with torch.cuda.graph(g):
            fn()
        res[name + "_capture"] = "ok"
    except cg.AttnError as e:
        res[name + "_capture"] = e.status
    fn()
    torch.cuda.synchronize()
    res[name + "_eager"] = cg.attn_device_check()
calls = dict(
    pack=lambda: cg.attn_pack4(k, v, k4, v4),
    fwd=lambda: cg.attn_prefill_window(q, k, v, 50),
    bwd=lambda: cg.attn_prefill_window_backward(q, k, v, o, lse, do, 50),
    win=lambda: cg.attn_decode_window(qd, k, v, lens, 50),
    four=lambda: cg.attn_decode4(qd, k4, v4, lens))
import sys
for name in sys.argv[1].split():
    in_capture(name, calls[name])
print(json.dumps(res))
"""


@pytest.mark.parametrize("names", ["fwd bwd win four", "pack", "four"])
def test_first_call_during_capture_is_refused(names):
    env = dict(os.environ, PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    r = subprocess.run([sys.executable, "-c", _FIRST_CALL, names], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    res = json.loads(r.stdout.strip().splitlines()[-1])
    for name in names.split():
        assert res[name + "_capture"] == ATTN_ERR_UNSUPPORTED, res
        assert res[name + "_eager"] == ATTN_OK, res

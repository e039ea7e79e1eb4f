"""The serving-step operators called in the ways that their header allows beside the plain ones:
from several host threads at once, at the sizes where a launch's resources change, on inputs that
only the kernels can refuse.  What each operator computes is tested in test_gpu_serving.py."""
import ctypes as C
import os
import subprocess
import sys
import textwrap
import threading

import numpy as np
import pytest

from oracle import serving

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def uw():
    import torch
    assert torch.cuda.is_available()
    from tests.conftest import build_library
    build_library()
    import decode_gemm_b200
    return decode_gemm_b200


def _at_once(*calls, times):
    """Run each call (a library function's status) `times` times, every one in a host thread of its own;
    the statuses that came back."""
    seen, start = set(), threading.Barrier(len(calls))

    def loop(call):
        start.wait(60)
        seen.update({call() for _ in range(times)})
    threads = [threading.Thread(target=loop, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return seen


def test_sample_from_several_host_threads(uw):
    """Vocabularies whose launches need different amounts of shared memory, on a stream each."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(1)
    cases = []
    for vocab in (100000, 900, 120000, 1100):
        x = torch.randn((75, vocab), generator=gen, device="cuda").to(torch.bfloat16)
        u, t = torch.rand(75, generator=gen, device="cuda"), torch.zeros(75, device="cuda")
        ids, stream = torch.zeros(75, dtype=torch.int64, device="cuda"), torch.cuda.Stream()
        a = uw.uw_sample_args(x.data_ptr(), u.data_ptr(), t.data_ptr(), None, None, None, ids.data_ptr(), None, 75, vocab, vocab, 1)
        cases.append((a, stream, ids, x, u, t))
    torch.cuda.synchronize()
    seen = _at_once(*(lambda a=a, s=s: uw.lib.uw_sample(C.byref(a), s.cuda_stream) for a, s, *_ in cases), times=5000)
    torch.cuda.synchronize()
    assert seen == {uw.UW_OK}
    for _, _, ids, x, *_ in cases:
        at = torch.arange(x.shape[1], device="cuda")
        assert torch.equal(ids, torch.where(x == x.amax(1, keepdim=True), at, x.shape[1]).amin(1))


def _plan_tensors(n):
    """One new token for each of n requests that store one already, as a uw_paged_plan_args."""
    import torch
    t = {k: torch.full((m,), v, dtype=d, device="cuda") for k, m, v, d in (
        ("ctx", n, 1, torch.int32), ("new", n, 1, torch.int32), ("head", 1, -7, torch.int32), ("table", n, 5, torch.int32),
        ("cu", n + 1, -7, torch.int32), ("kv", n, -7, torch.int32), ("pos", n, -7, torch.int32), ("slots", n, -7, torch.int64))}
    p = {k: v.data_ptr() for k, v in t.items()}
    return t, lambda uw: uw.uw_paged_plan_args(p["ctx"], p["new"], None, None, p["head"], p["table"], p["cu"], p["kv"],
                                               p["pos"], p["slots"], None, 1, n, n, 1, 0, 8)


def _plan_is_right(t, n):
    assert t["cu"].tolist() == list(range(n + 1)) and t["kv"].tolist() == [2] * n and t["head"].tolist() == [0]
    assert t["pos"].tolist() == [1] * n and t["slots"].tolist() == [5 * 8 + 1] * n


def test_plan_from_several_host_threads(uw):
    """Numbers of requests whose launches need different amounts of shared memory, on a stream each."""
    import torch
    cases = [(n, *_plan_tensors(n), torch.cuda.Stream()) for n in (8192, 3500, 7000, 4000)]
    torch.cuda.synchronize()
    seen = _at_once(*(lambda a=args(uw), s=s: uw.lib.uw_paged_plan(C.byref(a), s.cuda_stream) for _, _, args, s in cases),
                    times=5000)
    torch.cuda.synchronize()
    assert seen == {uw.UW_OK}
    for n, t, *_ in cases:
        _plan_is_right(t, n)


def _in_a_process(body):
    """Run `body` in a process that has launched nothing else before (limits and switches are per process)."""
    head = f"""
        import sys
        sys.path.insert(0, {ROOT!r})
        from tests import test_gpu_serving_calls as t
        import numpy as np
        import torch
        import decode_gemm_b200 as uw
    """
    return textwrap.dedent(head) + textwrap.dedent(body)


def _run(code, **env):
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, **env), capture_output=True, text=True, timeout=300,
                       cwd=ROOT)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_plan_around_the_shared_memory_that_needs_no_limit(uw):
    """From a few thousand requests on, a launch needs a raised limit; what the kernel holds beside the requests'
    numbers counts too.  Rising numbers in a process of its own, where no larger call has raised it."""
    out = _run(_in_a_process("""
        import ctypes as C
        for n in (3000, 3054, 3055, 3056, 3057, 3063, 3070, 3071, 3080):
            tensors, args = t._plan_tensors(n)
            status = uw.lib.uw_paged_plan(C.byref(args(uw)), None)
            assert status == uw.UW_OK, (n, status)
            torch.cuda.synchronize()
            t._plan_is_right(tensors, n)
        print("all planned")
    """))
    assert "all planned" in out


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (8, 8, 64)])
def test_attention_bounded_wait_reports_timeout(uw, heads, kv_heads, dim):
    """A wait on a signal that nothing gives runs out (100 ms here): the call raises UW_FLAG_TIMEOUT and returns, and
    the same process goes on attending.  The switch keeps back the last signal of units of two row tiles, so
    prompts run out and single tokens do not; it is read once per process, hence a process of its own."""
    out = _run(_in_a_process(f"""
        import time
        from tests import test_gpu_serving as g
        shape = ({heads}, {kv_heads}, {dim})
        prompts = g._requests(g._gen(1), np.random.default_rng(1), [(900, 700), (1500, 40), (800, 800), (64, 1)], 16, *shape)
        tokens = g._requests(g._gen(2), np.random.default_rng(2), [(300, 1), (1, 1), (0, 0), (2000, 1)], 16, *shape)
        for _ in range(3):
            began = time.monotonic()
            out, lse, flags = g._attend(uw, *prompts)
            assert flags == uw.UW_FLAG_TIMEOUT, flags
            assert time.monotonic() - began < 20
            assert bool((out[-3:] == 77).all()) and bool((lse[-3:] == 77).all())  # rows of no request
            g._check_attention(uw, *tokens)
        print("timeout reported, attention usable")
    """), UW_TEST_WITHHOLD_HANDOFF="1", UW_WAIT_LIMIT_MS="100")
    assert "timeout reported, attention usable" in out


def test_attention_reports_row_offsets_out_of_order(uw):
    """cu_q below zero, beyond the rows, or falling: reported, cut, and never followed."""
    from tests import test_gpu_serving as g
    gen, rng = g._gen(10), np.random.default_rng(10)
    q, kc, vc, table, cu, kv = g._requests(gen, rng, [(200, 2), (90, 1), (40, 40)], 16, 4, 2, 64)
    good, _, flag = g._attend(uw, q, kc, vc, table, cu, kv)
    assert flag == 0 and list(cu) == [0, 2, 3, 43] and q.shape[0] == 46
    for bad, sound in (([0, 2, 3, 47], 3), ([0, 2, 3, 2**31 - 1], 3), ([0, 2, 3, -2**31], 3), ([0, 2, 1, 1], 1),
                       ([-1, 2, 3, 43], 0), ([46, 46, 46, 45], 0)):
        out, _, flag = g._attend(uw, q, kc, vc, table, bad, kv)
        assert flag == uw.UW_FLAG_BAD_INPUT, bad
        assert np.array_equal(g._f64(out)[:sound], g._f64(good)[:sound]), bad
    # as far as the rows go, and requests without rows at their end: sound
    for fine in ([0, 2, 3, 46], [0, 2, 3, 3], [46, 46, 46, 46], [0, 0, 0, 0]):
        assert g._attend(uw, q, kc, vc, table, fine, kv)[2] == 0, fine


@pytest.mark.parametrize("heat", [1.0, 0.3, 5.0])
def test_sample_weights_to_what_is_stated(uw, heat):
    """Rows of two logits whose second weight lies within 2^-27 of min_p (which is a float, so 2^-25 apart at most),
    on either side: kept where it is larger, as long as the two are more than the stated 2^-29 apart.  (A table
    entry and a correction are each rounded to half a unit of at least 2^30: 2^-30 together; the correction's FP32
    steps, at most 2^-10 of the weight, add below 2^-32.)"""
    import torch
    rng, wide = np.random.default_rng(int(heat * 10)), np.longdouble
    top = rng.choice(np.float32([0, 7.25, -31.0, 18.6]), 1 << 20)
    low = (top - rng.uniform(0, 9, top.size) * heat).astype(np.float32)
    w = np.exp((low.astype(wide) - top.astype(wide)) / wide(np.float32(heat)))
    least = w.astype(np.float32)
    off = (w / least.astype(wide) - 1).astype(np.float64)
    rows = np.flatnonzero((np.abs(off) > 2.0**-29) & (np.abs(off) < 2.0**-27))[:60000]
    assert rows.size > 10000 and (off[rows] > 0).mean() > 0.3 and (off[rows] < 0).mean() > 0.3
    n = rows.size
    x = torch.from_numpy(np.stack([top[rows], low[rows]], 1)).cuda()
    # the last id that is kept: u is next to one, and its share is at least e^-9
    ids, u = torch.full((n,), -9, dtype=torch.int64, device="cuda"), torch.full((n,), 1 - 2.0**-24, device="cuda")
    uw.uw_sample(x, u, ids, temperature=torch.full((n,), heat, device="cuda"), min_p=torch.from_numpy(least[rows]).cuda())
    wrong = np.flatnonzero((ids.cpu().numpy() == 1) != (off[rows] > 0))
    assert wrong.size == 0, (wrong.size, np.log2(np.abs(off[rows][wrong])).tolist()[:9])


def test_calls_at_once_on_streams_and_in_graphs(uw):
    """Calls that share nothing, on a stream each, eager and as replayed graphs: what each gives alone."""
    import torch
    from tests import test_gpu_serving as g
    gen, rng = g._gen(40), np.random.default_rng(40)
    pieces = []
    for lens, heads, kv_heads, dim, window in (([(3000, 1), (70, 70), (0, 0), (5, 9)], 8, 2, 128, 0),
                                               ([(900, 300), (260, 1)], 6, 3, 64, 100), ([(40, 1)] * 200, 4, 4, 128, 0)):
        q, kc, vc, table, cu, kv = g._requests(gen, rng, lens, 16, heads, kv_heads, dim)
        t, c, l, out = g._ints(table), g._ints(cu), g._ints(kv), torch.zeros_like(q)
        ws = torch.empty(uw.uw_paged_attention_workspace_bytes(heads, kv_heads, dim), dtype=torch.uint8, device="cuda")
        pieces.append((out, lambda q=q, kc=kc, vc=vc, t=t, c=c, l=l, out=out, ws=ws, w=window:
                       uw.uw_paged_attention(q, kc, vc, t, c, l, out, window=w, ws=ws)))
    for rows, vocab in ((1, 131072), (200, 5003)):
        x, u, ids = torch.randn((rows, vocab), generator=gen, device="cuda") * 3, torch.rand(rows, generator=gen, device="cuda"), \
            torch.zeros(rows, dtype=torch.int64, device="cuda")
        p = torch.full((rows,), 0.95, device="cuda")
        pieces.append((ids, lambda x=x, u=u, ids=ids, p=p: uw.uw_sample(x, u, ids, top_p=p)))
    t, args = _plan_tensors(3500)
    plan = args(uw)
    pieces.append((t["slots"], lambda: uw._check(uw.lib.uw_paged_plan(C.byref(plan), torch.cuda.current_stream().cuda_stream), "plan")))
    want = []
    for out, call in pieces:
        call()
        torch.cuda.synchronize()
        want.append(out.clone())
    streams = [torch.cuda.Stream() for _ in pieces]
    graphs = []
    for out, call in pieces:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for graphed in (False, True):
        for out, _ in pieces:
            out.zero_()
        torch.cuda.synchronize()
        for i in range(20):
            for j, ((_, call), graph) in enumerate(zip(pieces, graphs)):
                with torch.cuda.stream(streams[(i + j) % len(pieces) if graphed and i % 5 == 0 else j]):
                    if graphed:
                        graph.replay()
                    else:
                        call()
            if graphed and i % 5 in (4, 0):  # (a graph moves to another stream only once its last run is over)
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        for k, ((out, _), w) in enumerate(zip(pieces, want)):
            assert torch.equal(out, w), (k, graphed)


def test_attention_keeps_bad_queries_to_their_rows(uw):
    """NaN and infinities in one row's query, and in rows of no request: every other row is bitwise as before."""
    import torch
    from tests import test_gpu_serving as g
    gen, rng = g._gen(50), np.random.default_rng(50)
    for heads, kv_heads, dim, window in ((8, 2, 128, 0), (6, 6, 64, 90), (16, 1, 128, 0)):
        q, kc, vc, table, cu, kv = g._requests(gen, rng, [(700, 300), (9, 1), (40, 1), (2000, 3), (0, 0)], 16, heads, kv_heads, dim)
        clean = g._attend(uw, q, kc, vc, table, cu, kv, window=window)
        last = int(cu[-1])
        for bad in (float("nan"), float("inf"), -float("inf")):
            rows = [0, 17, 299, 300, int(cu[3]) + 1]
            spoilt = q.clone()
            spoilt[rows] = bad
            spoilt[last:] = bad
            out, lse, flag = g._attend(uw, spoilt, kc, vc, table, cu, kv, window=window)
            others = [r for r in range(q.shape[0]) if r not in rows]
            assert flag == 0
            assert torch.equal(out[others], clean[0][others]) and torch.equal(lse[others], clean[1][others]), (heads, bad)
            assert bool(torch.isnan(out[rows]).all()), (heads, bad)

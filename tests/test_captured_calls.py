"""Calls captured into a HIP graph and replayed, with eager calls between the replays.

On the CPU, tests/host/capture_check.cpp is compiled host-only against the library's
ABI source, with stub kernel launchers and runtime calls, and run: what the step and
the orthogonalization enqueue on a stream that is being captured."""
import os
import shutil
import subprocess

import pytest
import torch

import newton_schulz_03_amd as nsa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "newton_schulz_03_amd", "csrc")
BF16, FP32 = torch.bfloat16, torch.float32


def _check(tmp_path, csrc):
    exe = tmp_path / "capture_check"
    build = subprocess.run(
        ["hipcc", "--offload-host-only", "-x", "hip", "-O1", "-std=c++17",
         "-I", os.path.join(ROOT, "include"), "-I", str(csrc),
         os.path.join(ROOT, "tests", "host", "capture_check.cpp"), "-o", str(exe)],
        capture_output=True, text=True, timeout=300)
    assert build.returncode == 0, build.stderr[-3000:]
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not found")
def test_captured_calls_copy_nothing(tmp_path):
    run = _check(tmp_path, CSRC)
    assert run.returncode == 0 and run.stdout.startswith("OK"), run.stdout + run.stderr


# (text in muon_abi.hip, its replacement, the failure the check must report)
PLANTED = [
    ("  if (capturing(stream)) return put_table(pl, ws, stream);\n", "", "copies nothing"),
    ("  if (capturing(stream)) return put_table(pl, ws, stream);\n",
     "  return put_table(pl, ws, stream);\n", "copies its table"),
    ("      if (capturing(s))\n", "      if (false)\n", "not refused"),
]


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not found")
@pytest.mark.parametrize("old,new,failure", PLANTED)
def test_planted_capture_mistakes_fail(tmp_path, old, new, failure):
    csrc = tmp_path / "csrc"
    shutil.copytree(CSRC, csrc)
    src = (csrc / "muon_abi.hip").read_text()
    assert src.count(old) == 1, old
    (csrc / "muon_abi.hip").write_text(src.replace(old, new))
    run = _check(tmp_path, csrc)
    assert run.returncode == 1 and failure in run.stdout, run.stdout + run.stderr


def replays(run, eager, pairs, change, times=4):
    """Captures run(), then replays it between eager calls and compares pairs()."""
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run()
    for k in range(times):
        change(k)
        eager()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in pairs():
            assert torch.equal(a, b), k


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,fp8_steps", [(BF16, 0), (BF16, 2), (FP32, 0)])
@pytest.mark.parametrize("batch", [3, 60])
def test_the_step_with_a_factor(batch, dtype, fp8_steps):
    shapes = [(64 + 33 * (i % 9), 200 + 71 * (i % 5)) for i in range(batch)]
    gen = torch.Generator().manual_seed(batch)
    ws, gs, ms = ([(torch.randn(s, generator=gen) * 1e-2).to(dtype).cuda() for s in shapes]
                  for _ in range(3))
    ws2, ms2 = [w.clone() for w in ws], [m.clone() for m in ms]
    factor = torch.full((1,), 0.5, device="cuda")
    room = nsa.allocate_workspace(shapes, dtype, "cuda", fp8=fp8_steps > 0)

    def change(k):
        factor.mul_(0.9)
        # a call that takes the staging slots, on other matrices
        nsa.step_batched(*([torch.randn((100 + k, 70), device="cuda").to(dtype)] for _ in range(3)))

    replays(lambda: nsa.step_batched(ws, gs, ms, grad_scale=factor, fp8_steps=fp8_steps, workspace=room),
            lambda: nsa.step_batched(ws2, gs, ms2, grad_scale=factor, fp8_steps=fp8_steps),
            lambda: zip(ws + ms, ws2 + ms2), change)


@pytest.mark.gpu
def test_the_plain_step_and_the_orthogonalization():
    gen = torch.Generator().manual_seed(9)
    xs = [torch.randn(s, generator=gen).to(BF16).cuda() for s in ((300, 700), (700, 301), (64, 64))]
    out, want = [torch.empty_like(x) for x in xs], [torch.empty_like(x) for x in xs]
    ms, ms2 = ([torch.zeros_like(x) for x in xs] for _ in range(2))
    ws, ws2 = ([torch.zeros_like(x) for x in xs] for _ in range(2))
    rooms = [nsa.allocate_workspace([tuple(x.shape) for x in xs], BF16, "cuda") for _ in range(2)]

    def run(w, o, m, rooms):
        nsa.ns_batched(xs, out=o, workspace=rooms[0])
        nsa.step_batched(w, xs, m, nesterov=True, workspace=rooms[1])

    def change(k):
        for x in xs:
            x.mul_(-1.25)

    replays(lambda: run(ws, out, ms, rooms), lambda: run(ws2, want, ms2, [None, None]),
            lambda: zip(out + ws + ms, want + ws2 + ms2), change)


def room(nbytes):
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device="cuda")
    return ws[(-ws.data_ptr()) % 256:]


def gradients(count):
    gen = torch.Generator().manual_seed(count)
    return [(torch.randn(100 + 131 * (i % 50), generator=gen) * 1e-3).to(FP32 if i % 3 else BF16).cuda()
            for i in range(count)]


@pytest.mark.gpu
@pytest.mark.parametrize("given", [True, False])  # a workspace of the caller's, or the graph's own
@pytest.mark.parametrize("count", [159, 160, 300])
def test_clip_into_other_buffers(count, given):
    # from 160 tensors on the table is written by kernels inside the graph
    gs = gradients(count)
    out, want = ([torch.zeros(g.shape, dtype=BF16, device="cuda") for g in gs] for _ in range(2))
    res, wres = torch.zeros(2, device="cuda"), torch.zeros(2, device="cuda")
    ws = room(nsa.grad_workspace_bytes([g.numel() for g in gs])) if given else None

    def change(k):
        for g in gs:
            g.mul_(0.7)

    replays(lambda: nsa.grad_clip_batched(gs, 1e-2, out=out, result=res, workspace=ws),
            lambda: nsa.grad_clip_batched(gs, 1e-2, out=want, result=wres),
            lambda: zip(out + [res], want + [wres]), change)


@pytest.mark.gpu
@pytest.mark.parametrize("count", [239, 240, 500])
def test_norm_and_clip_in_place(count):
    # from 240 tensors on the table is written by kernels inside the graph
    gs = gradients(count)
    twins = [g.clone() for g in gs]
    res, wres = torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")
    ws = [room(nsa.grad_workspace_bytes([g.numel() for g in gs])) for _ in range(2)]

    def run(ts, r, ws):
        nsa.grad_norm_batched(ts, max_norm=1.0, result=r[:2], workspace=ws[0])
        nsa.grad_clip_batched(ts, 1e-2, result=r[2:], workspace=ws[1])

    def change(k):
        for a, b in zip(gs, twins):
            a.mul_(1.7)
            b.mul_(1.7)

    replays(lambda: run(gs, res, ws), lambda: run(twins, wres, [None, None]),
            lambda: zip(gs + [res], twins + [wres]), change)


@pytest.mark.gpu
@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("count", [50, 51, 69, 70, 130])
def test_quantization_and_product(count, given):
    # from 70 matrices and 51 products on the tables are written by kernels inside the graph
    gen = torch.Generator().manual_seed(count)
    xs = [torch.randn((1 + 7 * (i % 11), 300), generator=gen).to(BF16).cuda() for i in range(count)]
    wq = nsa.f8_quantize_batched([torch.randn((136, 300), generator=gen).to(BF16).cuda()
                                  for _ in range(count)], block_rows=128)
    xq, xt, cs = ([[f(*x.shape) for x in xs] for _ in range(2)]
                  for f in (lambda r, c: nsa.f8_empty(r, c, "cuda"), lambda r, c: nsa.f8_empty(c, r, "cuda"),
                            lambda r, c: torch.zeros((r, 136), dtype=FP32, device="cuda")))
    ws = [room(nsa.f8_workspace_bytes(count)) if given else None for _ in range(2)]

    def run(k, ws):
        nsa.f8_quantize_batched(xs, transpose=True, out=xq[k], out_t=xt[k], workspace=ws[0])
        nsa.f8_matmul_batched(xq[k], wq, out=cs[k], accumulate=True, workspace=ws[1])

    def change(k):
        for x in xs:
            x.mul_(-1.5)

    def pairs():
        for a, b in zip(xq[0] + xt[0], xq[1] + xt[1]):
            yield a.q.view(torch.uint8), b.q.view(torch.uint8)
            yield a.scales, b.scales
        yield from zip(*cs)

    replays(lambda: run(0, ws), lambda: run(1, [None, None]), pairs, change)


@pytest.mark.gpu
def test_two_graphs_of_one_workspace():
    # one after the other on a stream: each writes its table at every replay
    a, b = gradients(300), gradients(280)
    ws = room(nsa.grad_workspace_bytes([g.numel() for g in a]))
    res = [torch.zeros(2, device="cuda") for _ in range(2)]
    graphs = []
    torch.cuda.synchronize()
    for gs, r in zip((a, b), res):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            nsa.grad_norm_batched(gs, max_norm=1e-3, result=r, workspace=ws)
        graphs.append(graph)
    for k in range(3):
        for g in a + b:
            g.mul_(1.1)
        want = [nsa.grad_norm_batched(gs, max_norm=1e-3) for gs in (a, b)]
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(res, want)), k

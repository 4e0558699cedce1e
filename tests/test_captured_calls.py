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

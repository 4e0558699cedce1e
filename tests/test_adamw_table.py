"""Where AdamW's table of tensors goes.

On the CPU, tests/host/adamw_table_check.cpp is compiled host-only against the
library's ABI source, with stub kernel launchers and runtime calls, and run; copies
of the source with planted mistakes must make it fail.  On the GPU, calls with a
table in the workspace, eager and captured."""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import newton_schulz_03_amd as nsa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "newton_schulz_03_amd", "csrc")


def _check(tmp_path, csrc):
    exe = tmp_path / "adamw_table_check"
    build = subprocess.run(
        ["hipcc", "--offload-host-only", "-x", "hip", "-O1", "-std=c++17",
         "-I", os.path.join(ROOT, "include"), "-I", str(csrc),
         os.path.join(ROOT, "tests", "host", "adamw_table_check.cpp"), "-o", str(exe)],
        capture_output=True, text=True, timeout=300)
    assert build.returncode == 0, build.stderr[-3000:]
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not found")
def test_one_copy_or_none(tmp_path):
    run = _check(tmp_path, CSRC)
    assert run.returncode == 0 and run.stdout.startswith("OK"), run.stdout + run.stderr


# (text in muon_abi.hip, its replacement, the failure the check must report)
PLANTED = [
    ("  if (capturing(s)) {", "  if (capturing(s) || true) {", "copies"),
    ("  if (capturing(s)) {", "  if (false) {", "copies"),
    ("      for (int32_t& x : prefix) x -= pl.prefix[i0];", "", "the prefixes do not span"),
]


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not found")
@pytest.mark.parametrize("old,new,failure", PLANTED)
def test_planted_table_mistakes_fail(tmp_path, old, new, failure):
    csrc = tmp_path / "csrc"
    shutil.copytree(CSRC, csrc)
    src = (csrc / "muon_abi.hip").read_text()
    assert src.count(old) == 1, old
    (csrc / "muon_abi.hip").write_text(src.replace(old, new))
    run = _check(tmp_path, csrc)
    assert run.returncode == 1 and failure in run.stdout, run.stdout + run.stderr


def state(numels, seed):
    g = torch.Generator().manual_seed(seed)
    return [[(torch.randn(n, generator=g) * s).to(dt).cuda() for n in numels]
            for s, dt in ((0.02, torch.bfloat16), (1e-3, torch.bfloat16), (1e-3, torch.float32))] + \
        [[(torch.randn(n, generator=g) * 1e-3).square().cuda() for n in numels]]


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [1024, 1025, 3000])
def test_many_small_tensors_equal_one_at_a_time(batch):
    # both ways to find a block's tensor, empty tensors among them
    rng = np.random.default_rng(batch)
    numels = [int(n) for n in rng.integers(0, 2500, batch)]
    numels[::9] = [0] * len(numels[::9])
    p, g, m, v = state(numels, batch)
    q, n, w = ([x.clone() for x in t] for t in (p, m, v))
    nsa.adamw_batched(p, g, m, v, step=2)
    for at in range(0, batch, 83):  # in tables that are arguments
        s = slice(at, at + 83)
        nsa.adamw_batched(q[s], g[s], n[s], w[s], step=2)
    for x, y in ((p, q), (m, n), (v, w)):
        assert all(torch.equal(a, b) for a, b in zip(x, y))


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [84, 1300])
def test_capture_and_replay(batch):
    numels = [100 + 37 * (i % 60) for i in range(batch)]
    p, g, m, v = state(numels, 7)
    q, n, w = ([x.clone() for x in t] for t in (p, m, v))
    s = torch.full((1,), 0.5, device="cuda")
    ws = torch.empty(nsa.adamw_workspace_bytes(numels) + 256, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        nsa.adamw_batched(p, g, m, v, step=2, grad_scale=s, workspace=ws)
    for k in range(4):
        s.mul_(0.9)
        # other calls use the staging slots, and the workspace, between replays
        nsa.adamw_batched(q, g, n, w, step=2, grad_scale=s)
        junk = state(numels[:90], 50 + k)
        nsa.adamw_batched(*junk, step=3, workspace=ws)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in ((p, q), (m, n), (v, w)):
            assert all(torch.equal(a, b) for a, b in zip(x, y)), k

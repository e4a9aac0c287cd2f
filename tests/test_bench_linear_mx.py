"""The benchmark's account of the pre-norm + MX linear step (CPU only)."""
import os
import subprocess
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

pytestmark = pytest.mark.cpu

T, K, N = 16384, 2048, 4096


@pytest.mark.parametrize("recipe,codes", [("mxfp4", 1024 + 64), ("mxfp8", 2048 + 64)])
def test_work(recipe, codes):
    fl, by = bench.linear_mx_work(T, K, N, recipe)
    assert set(fl.values()) == {2 * T * K * N} and len(fl) == 3
    # x, residual in, sum and y out: bf16; codes with scales; rstd; gamma
    assert by["add_rmsnorm"] == T * (4 * 2 * K + codes + 4) + 2 * K
    # dy, sum, the stream's gradient in, its gradient out; rstd; gamma
    assert by["add_rmsnorm_bwd"] == T * (4 * 2 * K + 4) + 2 * K
    for name in ("mx_linear", "add_rmsnorm", "add_rmsnorm_bwd", "add_rmsnorm_dgamma"):
        assert len(bench.source_hash(name)) == 16
    assert bench.LINEAR_PEAK == {"mxfp4": 10100.0, "mxfp8": 5000.0}


@pytest.mark.parametrize("recipe", ["mxfp4", "mxfp8"])
def test_oracle_sample(recipe):
    from precision_rl_amd import synth
    rng = np.random.Generator(np.random.PCG64(3))
    x, res, dout = (synth.normal_bf16(rng, (40, 256)) for _ in range(3))
    w, dy = synth.normal_bf16(rng, (136, 256)), synth.normal_bf16(rng, (40, 136))
    rec = bench.cpu_baseline_linear_mx(x, res, w, dy, dout, recipe, tokens=24)
    assert rec["value"] > 0 and rec["kind"] == "oracle" and "24 tokens" in rec["sample"]


@pytest.mark.parametrize("workload", ["learner", "qp"])
def test_mxfp8_is_refused_elsewhere(workload):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--workload", workload, "--recipe", "mxfp8"],
                       capture_output=True, text=True, timeout=120)
    assert r.returncode != 0 and "--workload linear" in r.stderr

"""How a 4-bit product of few tiles is cut (CTAs a tile, places of the ring, shared memory): a CTA with two stages or more has two places, so that one
is copied while the other is multiplied, and two CTAs fit an SM."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMS = 152
SM_BYTES, CTA_BYTES = 228 * 1024, 1024  # shared memory of an SM, and what a CTA takes beside its own
STATIC = 8 * (2 * 8 + 2) + 16 + 512     # barriers, the address of tensor memory, scales of the tokens


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    nvcc = next((c for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc") if c and os.path.exists(c)), None)
    if nvcc is None:
        pytest.skip("nvcc not found")
    exe = str(tmp_path_factory.mktemp("rule") / "fp4_rule")
    r = subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a", "-I", os.path.join(ROOT, "include"), "-I",
                        os.path.join(ROOT, "int4_weight_only_sgemv_gb300", "csrc"), os.path.join(ROOT, "tests", "host", "fp4_rule.cu"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr

    def of(calls):
        """calls: (block, tokens, rows, k)"""
        args, stages = [], []
        for block, tokens, rows, k in calls:
            x_tile = next(t for t in (8, 16, 32, 64, 128) if t >= tokens or t == 128)
            stage_k = 512 if x_tile <= 32 else 256
            stages.append(-(-(-(-k // 64) * 64) // stage_k))
            args += [block, x_tile, -(-rows // 128) * -(-tokens // 128), stages[-1], SMS]
        out = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=60)
        assert out.returncode == 0
        return [(n, *map(int, line.split())) for n, line in zip(stages, out.stdout.splitlines(), strict=True)]

    return of


def test_every_cta_has_two_places_and_two_fit_an_sm(plan):
    calls = [(block, tokens, rows, k) for block in (16, 32) for tokens in (1, 9, 17, 20, 32, 33, 64, 65, 128)
             for rows in (1, 129, 1000, 2048, 4096, 5120, 7680, 11008, 28672) for k in (64, 1000, 2048, 4096, 5000, 8192, 11008, 65536)]
    for call, (stages, split, ring, smem, stage, sent) in zip(calls, plan(calls), strict=True):
        most = -(-stages // split)  # of a CTA
        assert 1 <= split <= 8 and min(2, most) <= ring <= min(8, most), (call, split, ring)
        assert smem >= ring * stage
        late = call[1] > 32  # what is sent comes where the ring was
        tile = next(t for t in (8, 16, 32, 64, 128) if t >= call[1])
        assert smem >= (max(ring * stage, 512 * tile + sent) if late else max(ring * stage, 512 * tile) + sent)
        if smem > 112 * 1024:  # tiles of 128 tokens by 5 CTAs or more: one an SM
            assert tile == 128 and split > 4, (call, smem)
        else:
            assert 2 * (smem + STATIC + CTA_BYTES) <= SM_BYTES < 3 * (smem + CTA_BYTES), (call, smem)


def test_cases_that_are_split(plan):
    """The GPU tests' cases of 17 to 32 tokens are split by more than 4, with more stages a CTA than places."""
    import test_gpu_fp4_few as few
    calls = [(16, *c) for c in few.SPLIT]
    for call, (stages, split, ring, *_) in zip(calls, plan(calls), strict=True):
        assert split > 4 and stages // split > ring == 2, (call, stages, split, ring)


def test_clusters_of_every_size(plan):
    """The GPU tests' calls go to clusters of the sizes that they are named by."""
    import test_gpu_fp4_few as few
    for split, calls in few.CLUSTERS.items():
        assert [r[1] for r in plan([(16, *c) for c in calls])] == [split] * len(calls), split

"""Which attention kernel the GPU tests' cases go to: those meant for the chunk kernel have to reach it (and those meant for the
decode kernel not), whatever the thresholds become."""

import os
import shutil
import subprocess

import pytest

import test_gpu_kv_edges as edges

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMS = 152

# (dim, KV heads, query heads a KV head, requests as (tokens, new tokens)), as in the tests of the same names
CHUNK = {
    "large_chunks": (64, 1, 8, [(131, 131), (400, 140), (100, 135), (50, 1), (0, 0), (333, 9)]),
    "large_chunk_extreme_values": (128, 1, 8, [(200, 1), (190, 131)]),
    "large_chunk_scales": (128, 1, 8, [(330, 131), (260, 1)]),
    "large_chunk_rows_do_not_meet": (128, 1, 8, [(300, 131), (260, 4)]),
    "large_chunk_without_some_pages": (64, 1, 8, [(160, 131)]),
    "large_chunk_same_bits_and_far_offsets": (64, 8, 4, [(900, 300), (310, 270)]),
    "many_short_chunks": (128, 6, 4, [(n, n) for n in [33, 32, 1, 40, 65, 0, 34] * 3 + [64, 33, 50, 32, 36]]),
    "scores_past_24_bits": (128, 1, 8, [(300, 131), (40, 1)]),
    "large_chunk_rows_of_any_size": (64, 1, 8, [(190, 131), (60, 1)]),
    "windows_wider_than_any_length": (128, 1, 8, [(90, 131), (200, 1)]),
    "window_behind_freed_pages": (128, 1, 8, [(300 + a, 140) for a in (0, 9, 17, 31)]),
    "out_in_place_of_q": (128, 1, 8, [(300, 131), (50, 1)]),
    "many_requests_and_prompt_chunks 300": (64, 1, 8, edges.many_requests(300)),
    "many_requests_and_prompt_chunks 700": (64, 1, 8, edges.many_requests(700)),
    "many_requests_and_prompt_chunks 1400": (64, 1, 8, edges.many_requests(1400)),
    "prompts_of_many_rows": (128, 2, 8, edges.MANY_ROWS),
}
DECODE = {
    "rows_of_any_size": (64, 1, 8, [(90, 20), (140, 3)]),
    "prompts_of_many_rows 256": (256, 1, 8, edges.MANY_ROWS),
}


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    nvcc = next((c for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc") if c and os.path.exists(c)), None)
    if nvcc is None:
        pytest.skip("nvcc not found")
    exe = str(tmp_path_factory.mktemp("rule") / "kv_rule")
    r = subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a", "-I", os.path.join(ROOT, "include"), "-I",
                        os.path.join(ROOT, "int4_weight_only_sgemv_gb300", "csrc"), os.path.join(ROOT, "tests", "host", "kv_rule.cu"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr

    def of(dim, heads, ratio, reqs):
        args = (dim, heads, ratio, len(reqs), sum(n for _, n in reqs), max(n for _, n in reqs), SMS)
        return int(subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=60).stdout)

    return of


@pytest.mark.parametrize("name", CHUNK)
def test_cases_of_the_chunk_kernel(rule, name):
    dim, heads, ratio, reqs = CHUNK[name]
    rows = rule(dim, heads, ratio, reqs)
    assert rows > 0 and sum(n * ratio > rows for _, n in reqs) >= 1
    if name.startswith("many_requests"):
        assert sum(n * ratio > rows for _, n in reqs) > len(reqs) // 40  # every chunk among them


@pytest.mark.parametrize("name", DECODE)
def test_cases_of_the_decode_kernel(rule, name):
    assert rule(*DECODE[name]) == -1

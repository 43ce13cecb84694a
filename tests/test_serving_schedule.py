"""How paged_attention_kernel cuts its work into ranges, checked on the host: the kernel header's own
arithmetic, compiled for the CPU, over batches that would take too long to run."""
import os
import random
import subprocess

import pytest

from tensor_core_gemm_tcgen05_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))
KEYS_ALL, KEYS_OWN, KEYS_PREFIX, KEYS_BOTH = range(4)
SEQS_ALL, SEQS_SHORT, SEQS_LONG = range(3)


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("schedule") / "walk")
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17", "-I", os.path.join(_build.ROOT, "include"),
                    "-I", os.path.join(_build.PKG, "csrc"), "-o", exe, os.path.join(HERE, "schedule_walk.cu")], check=True)

    def run(tiles, group, kv_heads, seqs, keys=KEYS_ALL, which=SEQS_ALL, page=64, prefix=0, tile_tokens=None, grid=None):
        grid = (304 if tiles == 1 else 152) if grid is None else grid
        tile_tokens = 128 // group if tile_tokens is None else tile_tokens
        args = [tiles, group, kv_heads, page, prefix, keys, which, tile_tokens, grid] + [f"{n}:{kv}" for n, kv in seqs]
        p = subprocess.run([exe] + [str(a) for a in args], capture_output=True, text=True, timeout=600)
        assert p.stdout.startswith("ok "), (args[:9], seqs[:4], p.returncode, p.stdout)
        return [int(x) for x in p.stdout.split()[1:]]

    return run


# a head's units past 32 bits (and, in the middle one, past 2^32)
@pytest.mark.parametrize("group,tokens", [(128, 1_060_000), (64, 2_300_000), (8, 4_600_000)])
def test_prompts_whose_units_pass_32_bits(walk, group, tokens):
    assert walk(2, group, 1, [(tokens, tokens)])[1] > 2 ** 31


def test_long_prefix_under_many_tokens(walk):
    """Every tile of the tokens of all sequences reads the whole prefix."""
    assert walk(2, 8, 2, [(3000, 3000)] * 1000, keys=KEYS_PREFIX, page=1024, prefix=65536)[1] > 2 ** 31


def test_small_tiles_over_a_long_cache(walk):
    assert walk(1, 16, 1, [(2000, 2_000_000_000), (1, 7)])[1] > 2 ** 31


@pytest.mark.parametrize("group,kv", [(1, 100), (4, 2 ** 31 - 1024)])
def test_as_many_tokens_as_a_batch_may_have(walk, group, kv):
    """The last tile ends past them, the first new token stands far in front of the first key."""
    walk(2, group, 1, [(2 ** 31 - 1024, kv)], grid=3)


def test_random_batches(walk):
    rng = random.Random(5)
    for i in range(150):
        tiles, group, kv_heads = rng.choice([1, 2]), rng.choice([1, 2, 3, 5, 7, 8, 16, 100, 128]), rng.choice([1, 2, 5])
        page = rng.choice([16, 64, 1024])
        keys = rng.choice([KEYS_ALL, KEYS_OWN, KEYS_PREFIX] + ([KEYS_BOTH] if tiles == 1 else []))
        which = SEQS_ALL if keys >= KEYS_PREFIX else rng.choice([SEQS_ALL, SEQS_SHORT, SEQS_LONG])
        prefix = rng.choice([0, 1, 7, 40]) if keys == KEYS_ALL else rng.choice([1, 7, 40])
        tt = 128 // group if tiles == 2 else rng.randint(1, 128 // group)
        top = rng.choice([1, 4, 300])
        seqs = []
        for _ in range(rng.choice([1, 2, 9, 60, 400])):
            n = rng.randint(0, top)
            seqs.append((n, rng.choice([n, n + rng.randint(0, 50), rng.randint(0, 5000), 0])))
        walk(tiles, group, kv_heads, seqs, keys, which, page, prefix, tt, grid=rng.choice([1, 7, 152, 304]))

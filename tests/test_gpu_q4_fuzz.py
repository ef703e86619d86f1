"""Seeded random cases of the 4-bit operators on the GPU, through the automatic
choice of configuration, step and parts, against tests/q4_reference.py with
the tolerances of test_gpu_q4_weights.py and test_gpu_q4_cache.py."""
import random

import pytest

import tiled_dense_gemm_fp16_amd as g
from test_gpu_q4_cache import KINDS, check_append, check_attention
from test_gpu_q4_weights import EXPANDED, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(40))
def test_products(seed):
    r = random.Random(seed)
    m, n, k = (max(1, int(2 ** r.uniform(0, top))) for top in (8.5, 10, 12))
    if r.random() < 0.5:
        k = -(-k // 2) * 2
    config = r.choice([g.CONFIG_AUTO] * 3 + list(range(g.q4_num_configs())))
    group, shift = r.choice([32, 64, 128]), r.choice([0, 0, 1, 2, 8])
    try:
        g.plan_q4(m, n, k, group, config, A_ptr=2 * shift)
    except g.GemmError:
        config = g.CONFIG_AUTO                      # rows that the configuration does not take
    check(m, n, k, group, config=config, epilogue=r.choice(["none", "relu"]), alpha=r.choice([1.0, -0.3, 2.5]), shift=shift,
          seed=seed, splits=None if config == EXPANDED else r.choice([None, None, 1, 2, 5]))


@pytest.mark.parametrize("seed", range(60))
def test_attention(seed):
    r = random.Random(1000 + seed)
    dim, group = r.choice(KINDS)
    page, heads, ratio = r.choice([8, 16, 24, 32, 48, 64, 128]), r.choice([1, 2, 3]), r.choice([1, 1, 2, 3, 4, 5, 8, 9, 16, 20])
    batch = r.randint(1, 9)
    lengths = [r.choice([0, 1, page, page + 1, r.randint(0, 400)]) for _ in range(batch)]
    needed = sum(-(-n // page) for n in lengths)
    width = max(1, max(-(-n // page) for n in lengths))
    if r.random() < 0.6:
        width = max(width, r.choice([2048, 20000]) // page)          # room for steps of several blocks
    bad = [(b, r.randrange(-(-n // page)), r.choice([-1, needed + 3, 2 ** 31 - 1, -2 ** 31]))
           for b, n in enumerate(lengths) if n and r.random() < 0.3]
    check_attention(dim, group, page, lengths, heads * ratio, heads, pages=needed + 3, splits=r.choice([None, None, 1, 2, 5, 20]),
                    scale=r.choice([None, None, 0.2, -0.05]), bad=bad, width=width, max_length=r.choice([None, 1, 300]), seed=seed)


@pytest.mark.parametrize("seed", range(40))
def test_append(seed):
    r = random.Random(2000 + seed)
    dim, group = r.choice(KINDS)
    page, batch = r.choice([8, 16, 24, 40, 64]), r.randint(1, 7)
    past = [r.choice([0, 1, 7, 8, r.randint(0, 50)]) for _ in range(batch)]
    single = r.random() < 0.3
    new = [1] * batch if single else [r.choice([0, 1, 2, 9, r.randint(0, 30)]) for _ in range(batch)]
    pages = sum(-(-(p + n) // page) for p, n in zip(past, new))
    if pages > 60 or not sum(new):
        page, past, new = 64, [5] * batch, [1] * batch
    check_append(dim, group, page, past, new, heads=r.choice([1, 2, 5]), q_heads=r.choice([1, 4, 10]),
                 rotary=r.choice([0, 16, 32, dim, dim]), interleaved=r.random() < 0.5, single=single, fused=r.random() < 0.6,
                 tail=0 if single else r.choice([0, 3]), seed=seed)

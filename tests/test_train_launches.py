"""Launch shapes of the training-step operators at sizes that the header allows
(CPU checks): a launch of 2^32 threads or more in one dimension is refused by
the runtime, so no call may ask for one, and all rows have a block."""
import math

import pytest

from launch_records import launches

P = 0x10000  # a 16-byte aligned stand-in address: never dereferenced here
BIG = 1 << 60
LIMIT = 1 << 32


def topk(T, E=8, k=2):
    return "mxq_moe_topk", [P, 1, T, E, E, k, 0, P, P, None]


def topk_back(T, E=8, k=2):
    return "mxq_moe_topk_backward", [P, 1, T, E, E, P, k, 1, P, P, E, None]


def combine_back(T, C, k=1):
    return "mxq_moe_combine_backward", [P, 1, T, C, C, P, k, P, P, C, 16, P, C, P, None]


def loss(T, H, V):
    return "mxq_linear_cross_entropy", [P, H, P, H, P, T, H, V, P, P, P, BIG, None]


def loss_back(T, H, V):
    return "mxq_linear_cross_entropy_backward", [P, H, P, H, P, T, H, V, P, P, P, H, P, H, P, BIG, None]


def clip(chunks):
    return "mxq_clip_grad_norm", [P, 3, P, chunks, 1.0, P, P, None]


# (call, {part of a kernel's name: blocks of all its launches together})
CASES = [
    (topk(4), {"k_topk": 1}),
    (topk(8192, 256, 8), {"k_topk": 2048}),
    (topk((1 << 26) - 3), {"k_topk": 1 << 24}),
    (topk((1 << 26) + 5), {"k_topk": (1 << 24) + 2}),
    (topk(1 << 31, 256, 8), {"k_topk": 1 << 29}),
    (topk_back((1 << 26) + 5), {"k_topk_back": (1 << 24) + 2}),
    (combine_back(1 << 24, 2048), {"k_combine_back": 1 << 24}),
    (combine_back((1 << 24) + 3, 2048), {"k_combine_back": (1 << 24) + 3}),
    (combine_back((1 << 26) + 5, 64), {"k_combine_back": (1 << 24) + 2}),
    (loss((1 << 25) + 9, 64, 5), {"k_lse_join": (1 << 22) + 2}),
    (loss((1 << 22) + 300, 64, 1 << 17), {"k_lse_join": (1 << 19) + 38}),
    (loss_back((1 << 25) + 9, 512, 5), {"k_dx_join": ((1 << 25) + 9) // 2 + 1}),
    (loss_back(1 << 20, 16384, 5000), {"k_dx_join": 1 << 24}),
    (clip(1 << 20), {"k_clip_norm": 2048, "k_clip_scale": 1 << 20}),
    (clip((1 << 24) + 7), {"k_clip_norm": 2048, "k_clip_scale": (1 << 24) + 7}),
]


@pytest.fixture(scope="module")
def seen(tmp_path_factory):
    return launches(tmp_path_factory.mktemp("recorder"), [c for c, _ in CASES])


@pytest.mark.parametrize("n", range(len(CASES)), ids=[f"{c[0][4:]}-{'-'.join(str(a) for a in c[1] if isinstance(a, int) and a != P)}"
                                                      for c, _ in CASES])
def test_no_launch_reaches_the_runtimes_limit(seen, n):
    status, records = seen[n]
    assert status == 0
    assert records and all(r["launch"] for r in records)
    for r in records:
        assert all(g >= 1 for g in r["grid"])
        assert all(g * b < LIMIT for g, b in zip(r["grid"], r["block"])), r
    for name, blocks in CASES[n][1].items():
        mine = [math.prod(r["grid"]) for r in records if name + "I" in r["name"] or r["name"].count(f"{len(name)}{name}E")]
        assert sum(mine) == blocks, (name, mine)


def test_products_of_many_tokens_and_words_keep_all_their_tiles(tmp_path):
    """4194604 tokens x 131072 words: as many tiles in several launches as cover both."""
    (status, records), = launches(tmp_path, [loss((1 << 22) + 300, 64, 1 << 17)])
    assert status == 0
    products = [r for r in records if "k_loss_gemm" in r["name"]]
    sizes = {256: 256 * 256, 192: 192 * 256}
    covered = 0
    for r in products:
        assert "pipe" in r["name"]
        covered += math.prod(r["grid"]) * sizes[256 if "Li256E" in r["name"] else 192]
    assert covered >= ((1 << 22) + 300) << 17


def test_sorts_of_any_size_ask_for_one_amount_of_lds(tmp_path):
    """The limit on a kernel's dynamic LDS belongs to the kernel, not to a launch: a call that set its own size could
    lower it between another thread's setting and launch."""
    sort = lambda T, k, G: ("mxq_moe_sort", [P, T, k, G, P, P, P, P, BIG, None])
    calls = [sort(8192, 8, G) for G in (256, 512, 600, 1024, 1025, 2048, 4096)] + [sort(16, 8, 4096)]
    limits, largest = set(), 0
    for status, records in launches(tmp_path, calls):
        assert status == 0
        limits |= {r["lds"] for r in records if not r["launch"]}
        largest = max([largest] + [r["lds"] for r in records if r["launch"]])
        for i, r in enumerate(records):  # set before the launch that needs it
            assert not r["launch"] or r["lds"] <= 48 * 1024 or any(q["lds"] >= r["lds"] for q in records[:i]
                                                                   if not q["launch"])
    assert len(limits) == 1 and largest <= limits.pop() <= 160 * 1024 - 8320  # beside its static arrays

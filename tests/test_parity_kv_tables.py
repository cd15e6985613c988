"""Page tables, row starts, positions and slots made from lengths, against the
same made in Python (GPU tests)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from tests import step_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def check(lens, new, block, columns, pool, taken=0, rows=None, seed=0, behind=0, what=""):
    rng = np.random.default_rng(seed)
    seqs = len(lens)
    table = rng.integers(0, 1000, (seqs, columns)).astype(np.int32)
    if columns and seqs:
        table[rng.random(table.shape) < 0.1] = -1
    n = [min(max(0, int(a)), max(0, int(l))) for a, l in zip(new, lens)]
    rows = sum(n) + behind if rows is None else rows
    starts, positions, slots, after, want = ref.tables(table, lens, new, pool, taken, block, rows)
    t = torch.from_numpy(table).cuda()
    outs = [torch.full((rows,), 77, dtype=torch.int32).cuda(), torch.full((rows,), 77, dtype=torch.int64).cuda()]
    got = sg.kv_tables(t, gpu(lens), gpu(new), gpu(pool), gpu([taken]), block, rows, positions=outs[0], slots=outs[1])
    assert got[1] is outs[0] and got[2] is outs[1] and got[0].dtype == got[1].dtype == got[3].dtype == torch.int32
    assert np.array_equal(got[0].cpu().numpy(), starts), (what, "starts")
    k = len(positions)
    assert np.array_equal(got[1].cpu().numpy()[:k], positions) and (got[1][k:] == 77).all(), (what, "positions")
    assert np.array_equal(got[2].cpu().numpy()[:k], slots) and (got[2][k:] == 77).all(), (what, "slots")
    assert int(got[3]) == after, (what, "taken")
    assert np.array_equal(t.cpu().numpy(), want), (what, "table")


@pytest.mark.parametrize("block", [16, 128, 1024])
def test_small_batches(block):
    pool = np.arange(5000, 5400)
    for i, (lens, new) in enumerate([([1], [1]), ([0], [0]), ([16, 17, 33], [1, 1, 1]), ([0, 40, 0, 7], [0, 5, 0, 7]), ([130, 64, 31], [130, 20, 1]),
                                     ([16, 32, 48, 300], [16, 32, 1, 47]), ([5, 9, 2000], [0, 0, 0]), ([block, block + 1, 2 * block], [1, 1, block])]):
        check(lens, new, block, -(-max(lens) // block), pool, taken=i, seed=i, behind=i, what=(lens, new))


@pytest.mark.parametrize("seqs", [1, 63, 64, 65, 1023, 1024, 1025, 5000])
@pytest.mark.parametrize("most", [1, 40])
def test_many_sequences(seqs, most):
    print(f"[tables] {seqs} sequences, up to {most} new", flush=True)
    rng = np.random.default_rng(seqs + most)
    lens = rng.integers(0, 300, seqs)
    new = np.minimum(rng.integers(0, most + 1, seqs), lens)
    pool = rng.permutation(40 * seqs)
    check(lens, new, 16, 19, pool, taken=3, seed=seqs, behind=5)
    # Rows for some of them only, and for none.
    total = int(new.sum())
    check(lens, new, 16, 19, pool, rows=total // 2, seed=seqs)
    check(lens, new, 16, 19, pool, rows=0, seed=seqs)


@pytest.mark.parametrize("lens,new", [([20000], [20000]), ([16384, 1], [16384, 1]), ([16383, 1], [16383, 1]), ([9000, 0, 40000, 17, 30000], [9000, 0, 100, 17, 30000])])
def test_prompts(lens, new):
    pool = np.random.default_rng(1).permutation(10000)
    check(lens, new, 32, -(-max(lens) // 32), pool, taken=11)
    check(lens, new, 16, 100, pool, taken=0, behind=300, what="a table that is too short")
    check(lens, new, 16, 2500, pool[:700], taken=50, what="a pool that is too small")


@pytest.mark.parametrize("lens,new", [([8192], [8192]), ([8191, 1], [8191, 1]), ([8192, 5000], [8192, 1]), ([4096, 4099], [4096, 4095])])
def test_prompts_of_either_way(lens, new):
    # Rows up to where one work-group places them all, and the next one.
    print(f"[tables] {lens} {new}", flush=True)
    check(lens, new, 32, -(-max(lens) // 32), np.random.default_rng(2).permutation(1000), taken=3, behind=2)


def test_what_does_not_fit():
    # Pools that end before, between and after the call's pages, counters outside of them, tables without columns.
    lens, new, pool = [100, 37, 64, 5], [100, 1, 20, 5], np.arange(40, 60)
    for taken in (0, 8, 12, 19, 20, 1000, -3, 2**31 - 1, -(2**31)):
        check(lens, new, 16, 7, pool, taken=taken, what=taken)
    check(lens, new, 16, 7, pool[:0], what="an empty pool")
    check(lens, new, 16, 3, pool, what="few columns")
    check(lens, new, 16, 0, pool, what="no columns")
    check([], [], 16, 4, pool, taken=7, what="no sequences")
    check([], [], 16, 4, pool, taken=7, behind=20000, what="no sequences, rows behind")


def test_lengths_that_make_no_sense():
    pool = np.arange(100)
    check([-5, 10, -(2**31), 30], [3, 20, 1, -7], 16, 4, pool, what="negative lengths, more new than tokens, negative new")
    check([2**31 - 1, 50], [3, 50], 1024, 2**21, pool, what="the longest sequence")
    check([2**31 - 1, 2**31 - 1, 2**31 - 1], [0, 5, 1], 16, 3, pool, what="behind the table")


def test_sums_past_31_bits():
    # Two sequences whose new rows together pass 2^31: starts stop there, the rows that fit are placed.
    lens = [2**31 - 1, 2**31 - 1, 9]
    for rows in (100, 20000):
        table = torch.full((3, 2), 7, dtype=torch.int32).cuda()
        starts, positions, slots, after = sg.kv_tables(table, gpu(lens), gpu(lens), gpu([1, 2, 3]), gpu([0]), 1024, rows)
        assert starts.tolist() == [0, 2**31 - 1, 2**31 - 1, 2**31 - 1]
        assert torch.equal(positions.cpu(), torch.arange(rows, dtype=torch.int32))
        want = torch.tensor([1 if t < 1024 else 2 for t in range(min(rows, 2048))]) * 1024 + torch.arange(min(rows, 2048)) % 1024
        assert torch.equal(slots.cpu()[:2048], want) and (slots[2048:] == -1).all()
        assert table.tolist() == [[1, 2], [3, -1], [-1, 7]] and int(after) == 5


def test_in_place_and_repeated():
    # The counter in place, step after step: pages of one sequence do not meet another's.
    seqs, block, columns = 7, 16, 12
    rng = np.random.default_rng(3)
    pool = rng.permutation(200)
    table, taken = torch.full((seqs, columns), -1, dtype=torch.int32).cuda(), gpu([0])
    lens = np.zeros(seqs, np.int64)
    for step in range(9):
        new = rng.integers(0, 22, seqs)
        lens = lens + new
        got = sg.kv_tables(table, gpu(lens), gpu(new), gpu(pool), taken, block, int(new.sum()), taken_after=taken)
        assert got[3] is taken
        used = [-(-int(l) // block) for l in lens]
        t = table.cpu().numpy()
        pages = [int(p) for b, u in enumerate(used) for p in t[b, :u]]
        assert len(set(pages)) == len(pages) == int(taken) and set(pages) == set(pool[:len(pages)].tolist())
        assert all((t[b, u:] == -1).all() for b, u in enumerate(used))


def test_the_helper_refuses():
    table, lens, pool, one = torch.zeros(3, 4, dtype=torch.int32).cuda(), gpu([5, 6, 7]), gpu([1, 2, 3]), gpu([0])
    bad = {
        TypeError: [lambda: sg.kv_tables(table.long(), lens, lens, pool, one, 16, 3), lambda: sg.kv_tables(table, lens.long(), lens, pool, one, 16, 3),
                    lambda: sg.kv_tables(table, lens, lens, pool, one, 16, 3, slots=torch.zeros(3, dtype=torch.int32).cuda()),
                    lambda: sg.kv_tables(table[0], lens, lens, pool, one, 16, 3)],
        ValueError: [lambda: sg.kv_tables(table.cpu(), lens, lens, pool, one, 16, 3), lambda: sg.kv_tables(table, lens[:2], lens, pool, one, 16, 3),
                     lambda: sg.kv_tables(table, lens, lens[:2], pool, one, 16, 3), lambda: sg.kv_tables(table, lens, lens, pool, pool, 16, 3),
                     lambda: sg.kv_tables(table, lens, lens, pool.cpu(), one, 16, 3), lambda: sg.kv_tables(table, lens, lens, pool, one, 16, 3, starts=pool),
                     lambda: sg.kv_tables(table.t(), gpu([1] * 4), gpu([1] * 4), pool, one, 16, 3), lambda: sg.kv_tables(table, lens, lens, pool, one, 16, 2**31)],
        sg.SgemmError: [lambda: sg.kv_tables(table, lens, lens, pool, one, 48, 3), lambda: sg.kv_tables(table, lens, lens, pool, one, 8, 3),
                        lambda: sg.kv_tables(table, lens, lens, pool, one, 16, 3, positions=lens),
                        lambda: sg.kv_tables(table, lens, lens, pool, one, 16, 4, starts=(s := gpu([0] * 4)), positions=s)],
    }
    for error, calls in bad.items():
        for i, call in enumerate(calls):
            with pytest.raises(error):
                call()
                pytest.fail(f"{error.__name__} {i} was not refused")
    assert (table == 0).all()

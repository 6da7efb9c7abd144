"""engram_batch_plan against the scalar plan: exact, over admission by tokens and pages, finished and idle
requests, bad lengths and pages, and several steps that hand their lengths and pages on."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gpu_common import eg, say  # noqa: E402
from serving_common import plan_ref  # noqa: E402


def pool(rng, R, max_blocks, block_size, extra, fill=0.6):
    """Requests holding pages of a shuffled pool, and the stack of the rest."""
    cap = max_blocks * block_size
    held = (rng.random(R) * cap * fill).astype(np.int32)
    have = -(-held.astype(np.int64) // block_size)
    n_blocks = int(have.sum()) + extra
    order = rng.permutation(n_blocks).astype(np.int32)
    table = np.full((R, max_blocks), -7, np.int32)
    at = 0
    for r in range(R):
        table[r, :have[r]] = order[at:at + have[r]]
        at += have[r]
    free = np.full(n_blocks, -9, np.int32)
    free[:extra] = order[at:]
    return held, table, free, np.array([extra], np.int32), n_blocks


def run_and_check(lay, new, held, table, free, count, max_tokens):
    ref, table_ref, free_ref, errors = plan_ref(lay.block_size, lay.max_blocks, lay.n_blocks, new, held, table, free,
                                                count[0], max_tokens)
    dev = [torch.from_numpy(np.array(v, np.int32)).cuda() for v in (new, held, table, free, count)]
    plan = eg.BatchPlan(len(new), max_tokens)
    for f in eg.BatchPlan.FIELDS:
        getattr(plan, f).fill_(77)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for again in range(2):  # the inputs are not consumed: the same call gives the same plan
        err.zero_()
        eg.engram_batch_plan(lay, *dev, plan, err_count=err)
        torch.cuda.synchronize()
        for f in eg.BatchPlan.FIELDS:
            assert np.array_equal(getattr(plan, f).cpu().numpy(), np.array(ref[f])), (f, again)
        assert np.array_equal(dev[2].cpu().numpy(), table_ref) and np.array_equal(dev[3].cpu().numpy(), free_ref)
        assert int(err.item()) == errors
    return plan, ref, table_ref, free_ref


@pytest.mark.parametrize("R,block,max_blocks,extra,tokens", [
    (1, 16, 4, 2, 32), (3, 1, 40, 60, 100), (64, 16, 64, 200, 500), (257, 24, 30, 700, 4000), (1024, 16, 20, 900, 3000),
    (1025, 7, 9, 40, 2500), (4096, 64, 4, 6000, 20000)])
def test_plan_matches_the_scalar_plan(R, block, max_blocks, extra, tokens):
    say(f"[gpu] plan: {R} requests, pages of {block}, {tokens} tokens")
    for seed in range(3):
        rng = np.random.default_rng(100 * R + seed)
        held, table, free, count, n_blocks = pool(rng, R, max_blocks, block, extra)
        room = max_blocks * block - held
        new = np.minimum(rng.integers(0, max(2, 3 * tokens // R), R), room).astype(np.int32)
        new[rng.random(R) < 0.1] = -1
        lay = eg.make_page_layout(block, max_blocks, n_blocks)
        run_and_check(lay, new, held, table, free, count, tokens)


def test_refusals_keep_state_and_let_later_requests_in():
    say("[gpu] plan: out of tokens, out of pages, bad lengths, bad pages")
    lay = eg.make_page_layout(4, 3, 10)
    table = np.arange(27, dtype=np.int32).reshape(9, 3) % 10
    table[5, 0] = 10          # a page outside the pool
    table[5, 1] = -3
    free = np.array([9, 8, 7, 6, 5, 4, 3, 2, 1, 0], np.int32)
    #          grows  full  too long  negative  stays in its page  bad pages  needs 2  idle  decode in page
    new = np.array([1, 5, 9, 1, 2, 3, 8, 0, 1])
    held = np.array([0, 8, 4, -1, 1, 5, 0, 12, 6])
    for count in (3, 1, 0, -5, 99):
        for tokens in (30, 6, 0):
            run_and_check(lay, new, held, table, free, np.array([count]), tokens)


def test_released_pages_are_taken_again_in_the_same_step():
    say("[gpu] plan: pages of finished requests")
    lay = eg.make_page_layout(2, 4, 8)
    table = np.array([[0, 1, 2, 3], [4, 5, -1, -1], [6, -1, -1, -1]], np.int32)
    free = np.full(8, 7, np.int32)
    for held in ([8, 4, 2], [7, 3, 1], [0, 0, 0]):
        run_and_check(lay, [-1, 3, -4], held, table, free, np.array([1]), 16)
    # more pages given back than the list has entries
    run_and_check(eg.make_page_layout(2, 4, 8), [-1, -1, -1], [8, 4, 2], table, free, np.array([5]), 4)


def test_no_requests_or_no_tokens():
    say("[gpu] plan: nothing to plan")
    lay = eg.make_page_layout(16, 2, 4)
    z = np.zeros(0, np.int32)
    run_and_check(lay, z, z, np.zeros((0, 2), np.int32), np.arange(4, dtype=np.int32), np.array([4]), 5)
    run_and_check(lay, [0, -1], [0, 3], np.array([[0, 1], [2, 3]], np.int32), np.arange(4, dtype=np.int32), np.array([0]), 0)


def test_steps_hand_on_lengths_and_pages():
    say("[gpu] plan: 12 steps with two plans in turn")
    rng = np.random.default_rng(5)
    R, lay = 40, eg.make_page_layout(8, 12, 260)
    table = np.full((R, 12), -1, np.int32)
    free, held, count = rng.permutation(260).astype(np.int32), np.zeros(R, np.int32), 260
    t = [torch.from_numpy(v).cuda() for v in (table.copy(), free.copy())]
    plans = [eg.BatchPlan(R, 200), eg.BatchPlan(R, 200)]
    prev = plans[1]
    prev.free_left.fill_(260)
    for step in range(12):
        new = np.minimum(rng.integers(0, 12, R), 96 - held).astype(np.int32)
        new[rng.random(R) < 0.15] = -1
        ref, table, free, _ = plan_ref(8, 12, 260, new, held, table, free, count, 200)
        plan = plans[step & 1]
        eg.engram_batch_plan(lay, torch.from_numpy(new).cuda(), prev.seq_lens, t[0], t[1], prev.free_left, plan)
        for f in eg.BatchPlan.FIELDS:
            assert np.array_equal(getattr(plan, f).cpu().numpy(), np.array(ref[f])), (f, step)
        assert np.array_equal(t[0].cpu().numpy(), table) and np.array_equal(t[1].cpu().numpy(), free)
        held, count, prev = np.array(ref["seq_lens"], np.int32), ref["free_left"][0], plan
        # no page is held twice
        used = [int(p) for r in range(R) for p in table[r, :-(-int(held[r]) // 8)]] + [int(p) for p in free[:count]]
        assert sorted(used) == list(range(260))


def test_slots_past_32_bits():
    say("[gpu] plan: slots past 2^32")
    lay = eg.make_page_layout(1 << 20, 4, 1 << 16)
    free = np.zeros(1 << 16, np.int32)
    free[:3] = [65535, 5, 40000]
    plan, ref, _, _ = run_and_check(lay, [9, 4], [0, (1 << 20) - 2], np.array([[0] * 4, [65000] * 4], np.int32), free,
                                    np.array([3]), 16)
    assert max(ref["slots"]) > 1 << 32

"""The step's tables on the GPU: pkv_step_tables and pkv_release_blocks against
plain Python, exactly, with every array's other entries left as they were."""
import random

import pytest
import torch

import window_ref as ref
from paged_kv_cache_tables_gb300 import _binding as B
from paged_kv_cache_tables_gb300 import release_blocks, step_tables

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Pool:
    """Sequences of the given lengths with their blocks, and a shuffled free list."""

    def __init__(self, lens, max_blocks, spare, seed=0):
        rng = random.Random(seed)
        held = [-(-n // 16) for n in lens]
        ids = list(range(sum(held) + spare))
        rng.shuffle(ids)
        self.num_blocks = max(1, len(ids))
        self.table = []
        for n in held:
            self.table.append(ids[:n] + [-1] * (max_blocks - n))
            ids = ids[n:]
        self.lens, self.free, self.count = list(lens), ids + [-7] * 5, len(ids)

    def device(self, max_blocks):
        return (i32(self.lens), i32(self.table).reshape(len(self.lens), max_blocks), i32(self.free), i32([self.count]))


def run_step(pool, new, max_blocks, max_tokens, misaligned=False):
    lens, table, free, count = pool.device(max_blocks)
    S = len(pool.lens)
    ctx, cu = i32([-5] * (S + 1)), i32([-5] * (S + 2))
    o = 1 if misaligned else 0
    slots = torch.full((max_tokens + 2,), -9, dtype=torch.int64, device="cuda")
    pos = torch.full((max_tokens + 2,), -9, dtype=torch.int32, device="cuda")
    out, status = i32([-5]), i32([0])
    step_tables(lens, i32(new), table, free, count, pool.num_blocks, ctx[:S], cu[:S + 1], slots[o:max_tokens + o],
                pos[o:max_tokens + o], free_count_out=out, dev_status=status)
    assert ctx[S].item() == -5 and cu[S + 1].item() == -5
    edge = slice(0, 1) if misaligned else slice(max_tokens, None)
    assert (slots[edge] == -9).all() and (pos[edge] == -9).all() and slots[-1].item() == -9
    assert free.tolist() == pool.free and count.item() == pool.count and lens.tolist() == pool.lens
    return (table.tolist(), out.item(), ctx[:S].tolist(), cu[:S + 1].tolist(), slots[o:max_tokens + o].tolist(),
            pos[o:max_tokens + o].tolist()), status.item()


CASES = [
    ("one new token each, every place in a block", list(range(0, 40)), [1] * 40, 0),
    ("one sequence, one token", [0], [1], 0),
    ("one long chunk", [5], [3000], 7),
    ("idle sequences between", [0, 16, 31, 0, 48, 0], [0, 0, 17, 0, 1, 0], 3),
    ("nothing to do", [16, 0, 33], [0, 0, 0], 4),
    ("boundaries", [15, 16, 17, 0, 1, 32], [1, 16, 15, 16, 31, 33], 0),
    ("chunks and decodes", [100 * i for i in range(20)] + [7 * i for i in range(300)],
     [37 * i for i in range(20)] + [1] * 300, 1000),
]


@pytest.mark.parametrize("what,lens,new,pad", CASES, ids=[c[0] for c in CASES])
@pytest.mark.parametrize("misaligned", [False, True])
def test_step_tables(cuda_lib, what, lens, new, pad, misaligned):
    mb = 260
    pool = Pool(lens, mb, 900)
    T = sum(new) + pad
    got, status = run_step(pool, new, mb, T, misaligned)
    want = ref.step_tables(lens, new, pool.table, pool.free, pool.count, T)
    assert got == want and status == 0


@pytest.mark.parametrize("S", [255, 256, 257, 1024, 1025, 5000, B.TABLES_MAX_SEQS])
def test_step_tables_many_sequences(cuda_lib, S):
    rng = random.Random(S)
    lens = [rng.randint(0, 100) for _ in range(S)]
    new = [rng.choice([0, 1, 1, 1, rng.randint(2, 40)]) for _ in range(S)]
    need = sum(-(-(a + b) // 16) - -(-a // 16) for a, b in zip(lens, new))
    pool = Pool(lens, 9, need, seed=S)   # exactly enough
    T = sum(new)
    got, status = run_step(pool, new, 9, T)
    assert got == ref.step_tables(lens, new, pool.table, pool.free, pool.count, T) and status == 0
    assert got[1] == 0


@pytest.mark.parametrize("S", [21, 1537, 2100])
@pytest.mark.parametrize("misaligned", [False, True])
def test_step_tables_many_rows(cuda_lib, S, misaligned):
    """More rows than the launch has threads, few and many sequences, padding behind."""
    rng = random.Random(S)
    lens = [rng.randint(0, 100) for _ in range(S)]
    new = [1000 if s < 20 else rng.choice([0, 1, 5]) for s in range(S)]
    pool = Pool(lens, 70, 20 * 64 + S, seed=S)
    T = sum(new) + 1003
    got, status = run_step(pool, new, 70, T, misaligned)
    assert got == ref.step_tables(lens, new, pool.table, pool.free, pool.count, T) and status == 0


def test_step_tables_without_sequences(cuda_lib):
    pool = Pool([], 4, 3)
    got, status = run_step(pool, [], 4, 6)
    assert got == ([], 3, [], [0], [-1] * 6, [0] * 6) and status == 0


@pytest.mark.parametrize("lens,new,mb,spare,T,bit", [
    ([16, 5, 32], [1, 12, 1], 8, 2, 20, B.DEV_FREE_LIST),          # three blocks wanted, two there
    ([16, -1, 32], [1, 1, 1], 8, 9, 20, B.DEV_BAD_CONTEXT),
    ([16, 120, 32], [1, 9, 1], 8, 9, 20, B.DEV_BAD_CONTEXT),       # past the table
    ([16, 5, 2 ** 31 - 1], [1, 1, 2 ** 31 - 1], 8, 9, 20, B.DEV_BAD_CONTEXT),
    ([16, 5, 32], [1, -3, 1], 8, 9, 20, B.DEV_BAD_CHUNK),
    ([16, 5, 32], [10, 10, 1], 8, 9, 20, B.DEV_BAD_CHUNK),         # 21 tokens in 20 rows
    ([16, 5, 32], [1, 100, 1], 8, 9, 20, B.DEV_BAD_CHUNK),
])
def test_step_tables_takes_all_or_nothing(cuda_lib, lens, new, mb, spare, T, bit):
    pool = Pool([max(0, n) if n < 2 ** 20 else 0 for n in lens], mb, spare)
    pool.lens = lens
    got, status = run_step(pool, new, mb, T)
    assert status == bit
    assert got == (pool.table, pool.count, lens, [0] * 4, [-1] * T, [0] * T)


@pytest.mark.parametrize("count", [-1, 100000])
def test_step_tables_with_a_count_outside_the_list(cuda_lib, count):
    pool = Pool([3, 16], 4, 6)
    pool.count = count
    got, status = run_step(pool, [1, 1], 4, 4)
    assert status == B.DEV_FREE_LIST and got == (pool.table, count, [3, 16], [0] * 3, [-1] * 4, [0] * 4)


def test_step_tables_bad_block_ids_give_padding_slots(cuda_lib):
    pool = Pool([16, 5, 0], 4, 6)
    pool.free[pool.count - 1] = pool.num_blocks + 3   # the first id taken
    pool.table[1][0] = -1                             # an open block that is not there
    got, status = run_step(pool, [2, 1, 3], 4, 8)
    want = ref.step_tables(pool.lens, [2, 1, 3], pool.table, pool.free, pool.count, 8)
    assert status == B.DEV_BAD_BLOCK_ID
    assert got[:4] == want[:4] and got[5] == want[5]
    assert got[4] == [-1, -1, -1] + want[4][3:]


@pytest.mark.parametrize("S,chunk", [(5, 1), (700, 1), (2000, 9)])
def test_step_tables_in_place_and_replayed(cuda_lib, S, chunk):
    """context_lens written over seq_lens and the count in place, captured once
    and replayed: the loop a decode graph runs."""
    rng = random.Random(3)
    lens = [rng.randint(0, 50) for _ in range(S)]
    pool = Pool(lens, 16, S * 8)
    T = S * chunk
    seq, table, free, count = pool.device(16)
    new, cu, status = i32([chunk] * S), i32([0] * (S + 1)), i32([0])
    slots = torch.empty(T, dtype=torch.int64, device="cuda")
    pos = torch.empty(T, dtype=torch.int32, device="cuda")

    def call():
        step_tables(seq, new, table, free, count, pool.num_blocks, seq, cu, slots, pos, dev_status=status)

    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(7):
        g.replay()
    tab, n = pool.table, pool.count
    for _ in range(8):
        tab, n, lens, c, sl, ps = ref.step_tables(lens, [chunk] * S, tab, pool.free, n, T)
    assert status.item() == 0 and count.item() == n and seq.tolist() == lens and table.tolist() == tab
    assert slots.tolist() == sl and pos.tolist() == ps and cu.tolist() == c


# ---------------------------------------------------------------- release

def run_release(pool, mb, finished, window, sinks):
    lens, table, free, count = pool.device(mb)
    status = i32([0])
    release_blocks(table, lens, free, count, pool.num_blocks, finished=None if finished is None else i32(finished),
                   window=window, num_sinks=sinks, dev_status=status)
    return (table.tolist(), free.tolist(), count.item()), status.item()


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (16, 0), (17, 4), (31, 16), (32, 17), (100, 33), (4096, 4),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (5, 2 ** 31 - 1)])
@pytest.mark.parametrize("share", [0.0, 0.3, 1.0])
def test_release_blocks(cuda_lib, window, sinks, share):
    rng = random.Random(window + sinks)
    lens = list(range(0, 70)) + [rng.randint(0, 640) for _ in range(60)]
    pool = Pool(lens, 40, 5)
    for r in pool.table[::3]:   # some given back before
        r[2] = -1
    pool.free += [-7] * (len(lens) * 40)
    fin = [int(rng.random() < share) * rng.choice([1, -1, 7]) for _ in lens]
    got, status = run_release(pool, 40, fin, window, sinks)
    assert got == tuple(ref.release(pool.table, lens, fin, window, sinks, pool.free, pool.count, pool.num_blocks))
    assert status == 0


@pytest.mark.parametrize("S", [1, 16, 17, 32, 33, 100, 255, 256, 257, 3001, B.TABLES_MAX_SEQS])
def test_release_blocks_many_sequences(cuda_lib, S):
    rng = random.Random(S)
    lens = [rng.randint(0, 128) for _ in range(S)]
    pool = Pool(lens, 8, 3, seed=S)
    pool.free += [-7] * (S * 8)
    fin = [rng.randint(0, 1) for _ in lens]
    got, status = run_release(pool, 8, fin, 40, 4)
    assert got == tuple(ref.release(pool.table, lens, fin, 40, 4, pool.free, pool.count, pool.num_blocks))
    assert status == 0


@pytest.mark.parametrize("S", [3, 300])
def test_release_long_rows(cuda_lib, S):
    """Tables of many entries a row, with holes; a workspace of the caller's."""
    rng = random.Random(S)
    mb = 1000
    lens = [rng.randint(0, mb * 16) for _ in range(S)]
    pool = Pool(lens, mb, 3, seed=S)
    for r in pool.table:
        for j in rng.sample(range(mb), 300):
            r[j] = -1
    pool.free += [-7] * (S * mb)
    fin = [rng.randint(0, 1) for _ in lens]
    lens_d, table, free, count = pool.device(mb)
    work = torch.full((4 * S + 4,), 255, dtype=torch.uint8, device="cuda")
    status = i32([0])
    release_blocks(table, lens_d, free, count, pool.num_blocks, finished=i32(fin), window=5000, num_sinks=100,
                   workspace=work, dev_status=status)
    want = ref.release(pool.table, lens, fin, 5000, 100, pool.free, pool.count, pool.num_blocks)
    assert (table.tolist(), free.tolist(), count.item()) == tuple(want) and status.item() == 0


@pytest.mark.parametrize("S", [9, 300])
@pytest.mark.parametrize("mb,offset", [(333, 0), (334, 0), (335, 0), (336, 1), (336, 2), (336, 4)])
def test_release_rows_of_any_alignment(cuda_lib, S, mb, offset):
    rng = random.Random(mb + offset)
    lens = [rng.randint(0, mb * 16) for _ in range(S)]
    pool = Pool(lens, mb, 3, seed=S)
    for r in pool.table:
        for j in rng.sample(range(mb), 50):
            r[j] = -1
    pool.free += [-7] * (S * mb)
    fin = [int(rng.random() < 0.3) for _ in lens]
    lens_d, _, free, count = pool.device(mb)
    room = torch.full((offset + S * mb + 4,), -9, dtype=torch.int32, device="cuda")
    table = room[offset:offset + S * mb].view(S, mb)
    table.copy_(i32(pool.table))
    status = i32([0])
    release_blocks(table, lens_d, free, count, pool.num_blocks, finished=i32(fin), window=700, num_sinks=37, dev_status=status)
    want = ref.release(pool.table, lens, fin, 700, 37, pool.free, pool.count, pool.num_blocks)
    assert (table.tolist(), free.tolist(), count.item()) == tuple(want) and status.item() == 0
    assert (room[:offset] == -9).all() and (room[offset + S * mb:] == -9).all()


@pytest.mark.parametrize("S", [40, 400])
def test_release_captured_and_replayed(cuda_lib, S):
    """A loop step of two calls in a graph: grow by 16, give back what left a window of 40."""
    pool = Pool([5] * S, 40, S * 8)
    pool.free = pool.free[:pool.count] + [-7] * (S * 40)
    seq, table, free, count = pool.device(40)
    new, cu, status, none = i32([16] * S), i32([0] * (S + 1)), i32([0]), i32([0] * S)
    slots = torch.empty(S * 16, dtype=torch.int64, device="cuda")
    pos = torch.empty(S * 16, dtype=torch.int32, device="cuda")

    def call():
        step_tables(seq, new, table, free, count, pool.num_blocks, seq, cu, slots, pos, dev_status=status)
        release_blocks(table, seq, free, count, pool.num_blocks, finished=none, window=40, num_sinks=3, dev_status=status)

    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(20):
        g.replay()
    tab, fr, n, lens = pool.table, pool.free, pool.count, pool.lens
    for _ in range(21):
        tab, n, lens, _, sl, _ = ref.step_tables(lens, [16] * S, tab, fr, n, S * 16)
        tab, fr, n = ref.release(tab, lens, None, 40, 3, fr, n, pool.num_blocks)
    assert status.item() == 0 and count.item() == n and table.tolist() == tab and slots.tolist() == sl
    assert free.tolist()[:n] == fr[:n]


def test_release_without_finished_and_without_window_is_a_no_op(cuda_lib):
    pool = Pool([40, 3], 4, 3)
    got, status = run_release(pool, 4, None, 0, 4)
    assert got == (pool.table, pool.free, pool.count) and status == 0


@pytest.mark.parametrize("short", [0, 1])
def test_release_needs_room_for_all(cuda_lib, short):
    pool = Pool([40, 33, 20], 4, 3)
    pool.free = pool.free[:pool.count] + [-7] * (3 + 3 + 2 - short)
    fin = [1, 1, 1]
    got, status = run_release(pool, 4, fin, 0, 0)
    if short:
        assert status == B.DEV_FREE_LIST and got == (pool.table, pool.free, pool.count)
    else:
        assert status == 0
        assert got == tuple(ref.release(pool.table, pool.lens, fin, 0, 0, pool.free, pool.count, pool.num_blocks))


@pytest.mark.parametrize("count", [-1, 1000])
def test_release_with_a_count_outside_the_list(cuda_lib, count):
    pool = Pool([40, 33], 4, 3)
    pool.count = count
    got, status = run_release(pool, 4, [1, 0], 0, 0)
    assert status == B.DEV_FREE_LIST and got == (pool.table, pool.free, count)


def test_release_bad_ids_and_lengths(cuda_lib):
    pool = Pool([40, 33, 20], 4, 3)
    pool.free += [-7] * 12
    pool.table[0][1] = pool.num_blocks          # left where it is
    want = ref.release(pool.table, [40, 33, 0], [1, 1, 1], 0, 0, pool.free, pool.count, pool.num_blocks)
    pool.lens = [40, 33, -4]
    got, status = run_release(pool, 4, [1, 1, 1], 0, 0)
    assert status == B.DEV_BAD_BLOCK_ID | B.DEV_BAD_CONTEXT and got == tuple(want)
    pool.lens = [40, 33, 1000]                  # clamped to the table: 4 entries, 2 of them held
    want = ref.release(pool.table, [40, 33, 64], [1, 1, 1], 0, 0, pool.free, pool.count, pool.num_blocks)
    got, status = run_release(pool, 4, [1, 1, 1], 0, 0)
    assert status == B.DEV_BAD_BLOCK_ID | B.DEV_BAD_CONTEXT and got == tuple(want)


def test_step_then_release_on_a_side_stream_with_padding_rows(cuda_lib):
    """Two calls in a row on a stream of their own, the second taking what the
    first wrote; ids come back in the order the next step takes them."""
    pool = Pool([0, 30, 64], 8, 10)
    seq, table, free, count = pool.device(8)
    new, cu, status = i32([20, 3, 1]), i32([0] * 4), i32([0])
    slots = torch.empty(32, dtype=torch.int64, device="cuda")
    pos = torch.empty(32, dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    fin = i32([0, 1, 0])
    step_tables(seq, new, table, free, count, pool.num_blocks, seq, cu, slots, pos, dev_status=status, stream=st)
    release_blocks(table, seq, free, count, pool.num_blocks, finished=fin, window=20, num_sinks=4, dev_status=status,
                   stream=st)
    st.synchronize()
    tab, n, lens, _, sl, ps = ref.step_tables([0, 30, 64], [20, 3, 1], pool.table, pool.free, pool.count, 32)
    assert slots.tolist() == sl and pos.tolist() == ps
    tab, fr, n = ref.release(tab, lens, [0, 1, 0], 20, 4, pool.free, n, pool.num_blocks)
    assert table.tolist() == tab and free.tolist()[:n] == fr[:n] and count.item() == n and status.item() == 0


def test_release_of_many_rows_on_a_given_stream(cuda_lib):
    """Its workspace is the given stream's memory: what the current stream takes meanwhile is another's."""
    rng = random.Random(8)
    S, mb = 2000, 64
    lens = [rng.randint(0, mb * 16) for _ in range(S)]
    pool = Pool(lens, mb, 3)
    pool.free += [-7] * (S * mb)
    fin = [rng.randint(0, 1) for _ in lens]
    lens_d, table, free, count = pool.device(mb)
    status, fin_d, st = i32([0]), i32(fin), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    release_blocks(table, lens_d, free, count, pool.num_blocks, finished=fin_d, window=100, num_sinks=4, dev_status=status,
                   stream=st)
    others = [torch.full((4 * S + 4,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.current_stream().wait_stream(st)
    want = ref.release(pool.table, lens, fin, 100, 4, pool.free, pool.count, pool.num_blocks)
    assert (table.tolist(), free.tolist(), count.item()) == tuple(want) and status.item() == 0
    assert all((o == 255).all() for o in others)

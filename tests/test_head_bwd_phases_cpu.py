"""The barriers of the per-head scan's bf16 backward (head_mma_bwd.cu, head_bwd_kernel),
as a model on the host: its warps' waits and arrivals in random interleavings, a barrier
seen through a phase's parity only, as the hardware shows it. Every reader has to find the
panel that it asks for, no writer may cover what is still read, and every warp has to come
to its end, for heads of one to four panels and any number of heads in a CTA."""

import random

import pytest

WORKERS, FINISHERS = 4, 2  # of 16 and 2 warps; half of the workers take <S0, dS> as well


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):
        """What a wait for this parity sees: the running phase has the other one."""
        return (self.phase & 1) != (parity & 1)


class Place:
    """A buffer that `writers` fill for a panel and `readers` read; one panel at a time."""

    def __init__(self, name, writers, readers):
        self.name, self.writers, self.readers = name, writers, readers
        self.panel, self.wrote, self.read = -1, writers, readers

    def write(self, panel):
        if panel != self.panel:
            assert self.wrote == self.writers and self.read == self.readers, \
                f"{self.name}: panel {panel} covers panel {self.panel} in use"
            self.panel, self.wrote, self.read = panel, 0, 0
        self.wrote += 1

    def use(self, panel):
        assert self.panel == panel and self.wrote == self.writers, f"{self.name}: read for panel {panel}, holds {self.panel}"
        self.read += 1


class Stuck(AssertionError):
    pass


def run(heads, np_, seed, every_panel=True):
    """One CTA with `heads` heads of np_ panels. every_panel: both finishing warps wait for every
    panel's sums and free them; otherwise each passes over the other one's panels without a
    wait, and one arrival frees a panel's sums."""
    rng, count = random.Random(seed), heads * np_
    b = dict(ss=Barrier(1), ss_free=Barrier(WORKERS // 2 + 1), dm=Barrier(1), vy=Barrier(1), mt=Barrier(WORKERS), du=Barrier(1))
    for i in range(2):
        b["ud", i], b["epi", i] = Barrier(1), Barrier(WORKERS)
        b["fin", i] = Barrier(FINISHERS if every_panel else 1)
    sums = [Place(f"sums {i}", WORKERS, 1) for i in range(2)]
    # u, dy and tables: dM, every worker twice (tables, then rows), the product for du, the store
    ud = [Place(f"u, dy {i}", 1, 1 + 2 * WORKERS + 1 + 1) for i in range(2)]
    states = Place("S0, dS", 1, WORKERS // 2 + 1)
    dm, m_t = Place("dM", 1, WORKERS), Place("M", WORKERS, 1)
    vy, du = Place("V, Yi", 1, WORKERS), Place("du", 1, WORKERS)
    copies, products = [], []  # under way: copies end in any order, products in theirs

    def loader():
        for it in range(count + 2):
            if 2 <= it < count + 2:
                yield b["epi", it & 1], (it >> 1) - 1
                ud[it & 1].use(it - 2)
            if it >= count:
                continue
            copies.append(lambda it=it: (ud[it & 1].write(it), b["ud", it & 1].arrive()))
            if it > 0:
                yield b["ss_free"], it - 1
            copies.append(lambda it=it: (states.write(it), b["ss"].arrive()))

    def issuer():
        def issue_dm(it):
            products.append(lambda: (ud[it & 1].use(it), dm.write(it), b["dm"].arrive()))

        yield b["ud", 0], 0
        issue_dm(0)
        for it in range(count):
            yield b["ss"], it
            if it > 0:
                yield b["epi", (it - 1) & 1], (it - 1) >> 1
            products.append(lambda it=it: (states.use(it), vy.write(it), b["vy"].arrive(), b["ss_free"].arrive()))
            yield b["mt"], it
            products.append(lambda it=it: (m_t.use(it), ud[it & 1].use(it), du.write(it), b["du"].arrive()))
            if it + 1 < count:
                yield b["ud", (it + 1) & 1], (it + 1) >> 1
                issue_dm(it + 1)

    def worker(w):
        for it in range(count):
            if w >= WORKERS // 2:
                yield b["ss"], it
                states.use(it)
                b["ss_free"].arrive()
            if it >= 2:
                yield b["fin", it & 1], (it >> 1) - 1
            yield b["ud", it & 1], it >> 1
            ud[it & 1].use(it)
            yield b["dm"], it
            dm.use(it)
            m_t.write(it)
            b["mt"].arrive()
            yield b["vy"], it
            vy.use(it)
            yield b["du"], it
            du.use(it)
            ud[it & 1].use(it)
            sums[it & 1].write(it)
            b["epi", it & 1].arrive()

    def finisher(f):
        for it in range(count):
            mine = it // np_ % FINISHERS == f
            if not mine and not every_panel:
                continue
            yield b["epi", it & 1], it >> 1
            if mine:
                sums[it & 1].use(it)
            b["fin", it & 1].arrive()

    warps = [loader(), issuer()] + [worker(w) for w in range(WORKERS)] + [finisher(f) for f in range(FINISHERS)]
    waits = {i: next(w, None) for i, w in enumerate(warps)}
    waits = {i: q for i, q in waits.items() if q is not None}
    pace = [rng.random() ** 2 + 0.01 for _ in warps]  # some warps are slow throughout
    while waits or copies or products:
        ready = [i for i, (bar, parity) in waits.items() if bar.passed(parity)]
        if not ready and not copies and not products:
            raise Stuck(f"{len(waits)} warps wait for good")
        kinds = [(pace[i], i) for i in ready] + [(0.3, "copy")] * bool(copies) + [(0.3, "product")] * bool(products)
        pick = rng.choices([k for _, k in kinds], [p for p, _ in kinds])[0]
        if pick == "copy":
            copies.pop(rng.randrange(len(copies)))()
        elif pick == "product":
            products.pop(0)()
        else:
            nxt = next(warps[pick], None)
            if nxt is None:
                del waits[pick]
            else:
                waits[pick] = nxt
    for place in (*sums, *ud, states, dm, m_t, vy, du):
        assert place.wrote == place.writers and place.read == place.readers, place.name


@pytest.mark.parametrize("np_", [1, 2, 3, 4])
def test_every_panel_is_read_once_and_every_warp_ends(np_):
    for heads in range(1, 9):
        for seed in range(25):
            run(heads, np_, seed)


@pytest.mark.parametrize("np_", [2, 3, 4])
def test_model_sees_skipped_phases(np_):
    """Finishing warps that pass over the other one's panels take an older phase for theirs:
    the model has to show it with two heads and more, and with one head, or heads of one
    panel, not."""
    for heads in (2, 3, 4, 6):
        with pytest.raises(AssertionError):
            for seed in range(25):
                run(heads, np_, seed, every_panel=False)
    for seed in range(25):
        run(1, np_, seed, every_panel=False)
        run(5, 1, seed, every_panel=False)

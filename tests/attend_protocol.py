"""A model of the attention kernel's warps, barriers, copies and products, for the CPU.

The kernel's roles (scheduler, copy producer, product issuer, softmax and output warps) hand
row blocks, ring stages, queries and accumulators to one another by barriers. Here each role is
a generator with the kernel's waits and arrivals in the kernel's order, copies and products
finish at random times, and every wait may give up, as it does when it runs out. A trial raises
Fault for what would be undefined on the device: an arrival beyond a phase's count, a copy into
a stage that is being filled or read, a product of a stage that has not landed, partial results
over a stage being filled, work in flight when the CTA exits, a call that does not end."""

from __future__ import annotations

import random


class Fault(Exception):
    pass


class Barrier:
    """An mbarrier: a phase ends when all its arrivals and expected bytes are in."""

    def __init__(self, count, name):
        self.count = self.pending = count
        self.tx = self.phase = 0
        self.name = name

    def _advance(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def arrive(self, expect=0):
        if self.pending == 0:
            raise Fault(f"{self.name}: arrival beyond the phase's count")
        self.pending -= 1
        self.tx += expect
        self._advance()

    def complete(self):
        self.tx -= 1
        self._advance()

    def over(self, parity):
        return (self.phase & 1) != parity


class Cta:
    """One CTA: `blocks` are (key tiles, row tiles) of the row blocks it may take; a persistent
    one takes them one by one, a cluster's only has one. `mistakes` leaves out what the kernel
    does against a fault: "drain" (the copies and products that a role waits for before it
    ends, also if another role gives up later), "hand back" (a stage is only given back when
    its products are issued)."""

    def __init__(self, rng, row_tiles, stages, blocks, cluster, give_up, mistakes=()):
        self.rng, self.nq, self.stages, self.cluster = rng, row_tiles, stages, cluster
        self.give_up, self.mistakes = give_up, mistakes
        self.blocks, self.taken_block = list(blocks), None
        self.output_warps = row_tiles == 2
        w = self.warps = 4 if self.output_warps else rng.choice([1, 2, 4])  # with rows, per row tile
        tiles = range(row_tiles)
        self.full = [Barrier(1, f"full[{i}]") for i in range(stages)]
        self.empty = [Barrier(1, f"empty[{i}]") for i in range(stages)]
        self.qfull, self.qempty, self.sfull, self.ofull = ([Barrier(1, n) for _ in tiles]
                                                           for n in ("qfull", "qempty", "sfull", "ofull"))
        self.pfull = [[Barrier(w, "pfull"), Barrier(w, "pfull")] for _ in tiles]
        self.ofree, self.rfull = [Barrier(w, "ofree") for _ in tiles], [Barrier(w, "rfull") for _ in tiles]
        self.staged, self.unstaged = [Barrier(w, "staged") for _ in range(2)], [Barrier(1, "unstaged") for _ in range(2)]
        self.wfull = [Barrier(1, "wfull") for _ in range(2)]
        self.wempty = [Barrier((row_tiles + (1 if self.output_warps else 0)) * w + 2, "wempty") for _ in range(2)]
        self.want, self.taken, self.done = Barrier(1, "want"), Barrier(1, "taken"), Barrier(1, "done")
        self.abort = False
        self.work = [None, None]
        self.copies = []   # completions to come, in any order
        self.tensor = []   # (what a product reads, or the barrier of a commit), in order
        self.filling = {}  # stage -> halves of a tile to come

    # ------------------------------------------------------------ waits
    def wait(self, bar, parity):
        while not bar.over(parity):
            if not self.abort and self.rng.random() < self.give_up:
                self.abort = True
            if self.abort:
                return False
            yield
        return True

    def drain(self, bar, parity):
        while not bar.over(parity):
            yield

    def next_work(self, count):
        slot = count & 1
        if not (yield from self.wait(self.wfull[slot], (count >> 1) & 1)):
            return None
        w = self.work[slot]
        yield
        self.wempty[slot].arrive()
        return w

    # ------------------------------------------------------------ roles
    def scheduler(self):
        n = tries = 0
        item, ok = self.blocks.pop(0), True

        def publish(w):
            nonlocal n
            if n >= 2 and not (yield from self.wait(self.wempty[n & 1], ((n >> 1) - 1) & 1)):
                return False
            self.work[n & 1] = w
            self.wfull[n & 1].arrive()
            n += 1
            return True

        def answer():
            self.taken_block = self.blocks.pop(0) if self.blocks else None
            self.taken.complete()

        while True:
            ok = yield from publish(item)
            if ok and not self.cluster:
                ok = yield from self.wait(self.want, (n - 1) & 1)
            if not ok or self.cluster:
                break
            self.taken.arrive(expect=1)
            self.copies.append(answer)
            if not (yield from self.wait(self.taken, tries & 1)):
                ok = False
                yield from self.drain(self.taken, tries & 1)
                break
            tries += 1
            item = self.taken_block
            if item is None:
                break
        if ok:
            yield from publish(())

    def copy_in(self, stage):
        if self.filling.get(stage):
            raise Fault("copy into a stage that is being filled")
        if any(stage in what for what in self.tensor if isinstance(what, tuple)):
            raise Fault("copy into a stage that is being read")
        self.full[stage].arrive(expect=2)
        self.filling[stage] = 2

        def landed():
            self.filling[stage] -= 1
            self.full[stage].complete()
        self.copies += [landed, landed]

    def producer(self):
        st = ph = g = works = 0
        loads, ok = [0, 0], True
        while ok:
            w = yield from self.next_work(works)
            works += 1
            if not w:
                break
            tiles, nq = w
            for i in range(2 * tiles):
                if i == max(2 * tiles - 8, 0):
                    self.want.arrive()
                if g >= self.stages:
                    ok = yield from self.wait(self.empty[st], ph ^ 1)
                if not ok:
                    break
                yield
                self.copy_in(st)
                g += 1
                st += 1
                if st == self.stages:
                    st, ph = 0, ph ^ 1
                for q in range(nq if i == 0 else 0):
                    if loads[q] > 0:
                        ok = yield from self.wait(self.qempty[q], (loads[q] - 1) & 1)
                    if not ok:
                        break
                    loads[q] += 1
                    if any(("q", q) in what for what in self.tensor if isinstance(what, tuple)):
                        raise Fault("copy over queries that are being read")
                    self.qfull[q].arrive(expect=2)
                    self.copies += [self.qfull[q].complete] * 2
                    yield
                if not ok:
                    break
        if "drain" in self.mistakes and not self.abort:
            return
        for q in range(self.nq):
            if loads[q] > 0:
                yield from self.drain(self.qfull[q], (loads[q] - 1) & 1)
        for s in range(min(self.stages, g)):
            yield from self.drain(self.full[s], ph if s < st else ph ^ 1)

    def product(self, *what):
        if any(self.filling.get(x) for x in what):
            raise Fault("product of a stage that has not landed")
        self.tensor.append(what)

    def issuer(self):
        works = loads = tiles = outs = seen = st = ph = nt = nq = sv = 0
        ok, issued = True, False
        bits = lambda n: 3 if n == 2 else 1

        def step():
            nonlocal st, ph
            st += 1
            if st == self.stages:
                st, ph = 0, ph ^ 1

        while True:
            w = yield from self.next_work(works)
            works += 1
            more = bool(w) and w[0] > 0
            nq1 = w[1] if more else 0
            for q in range(self.nq):
                if q < nq:
                    parity = ((tiles >> q) ^ (nt - 1)) & 1
                    for half in range(2):
                        ok = yield from self.wait(self.pfull[q][half], parity)
                        if not ok:
                            break
                        self.product(sv)
                        yield
                    if not ok:
                        break
                    self.tensor.append(self.ofull[q])
                if q < nq1:
                    ok = q > 0 or (yield from self.wait(self.full[st], ph))
                    ok = ok and (yield from self.wait(self.qfull[q], (loads >> q) & 1))
                    if not ok:
                        break
                    issued = True
                    self.product(st, ("q", q))
                    self.tensor.append(self.sfull[q])
                    if w[0] == 1:
                        self.tensor.append(self.qempty[q])
                    yield
            if not ok:
                break
            if nq > 0:
                self.tensor.append(self.empty[sv])
            if nt & 1:
                tiles ^= bits(nq)
            if not more:
                break
            self.tensor.append(self.empty[st])
            nt, nq = w
            loads ^= bits(nq)
            step()
            sv = st
            ok = yield from self.wait(self.full[sv], ph)
            for q in range(nq):
                if ok and (seen >> q) & 1:
                    ok = yield from self.wait(self.ofree[q], ((outs >> q) & 1) ^ 1)
            seen |= bits(nq)
            outs ^= bits(nq)
            for j in range(nt - 1):
                if not ok:
                    break
                step()
                sk, pk = st, ph
                step()
                for q in range(nq):
                    parity = ((tiles >> q) ^ j) & 1
                    ok = yield from self.wait(self.pfull[q][0], parity)
                    if not ok:
                        break
                    self.product(sv)
                    yield
                    ok = yield from self.wait(self.pfull[q][1], parity)
                    if not ok:
                        break
                    self.product(sv)
                    if q == 0:
                        ok = yield from self.wait(self.full[sk], pk)
                    self.product(sv)
                    if q == nq - 1:
                        self.tensor.append(self.empty[sv])
                    if not ok:
                        break
                    self.product(sk, ("q", q))
                    yield
                    if q == nq - 1:
                        ok = yield from self.wait(self.full[st], ph)
                    self.product(sk, ("q", q))
                    self.tensor.append(self.sfull[q])
                    if j + 2 == nt:
                        self.tensor.append(self.qempty[q])
                if not ok and "hand back" not in self.mistakes:
                    break
                self.tensor.append(self.empty[sk])
                sv = st
            if not ok:
                break
            step()
            if self.filling.get(sv):
                raise Fault("zeroing rows of a stage that has not landed")
        if issued and ("drain" not in self.mistakes or not ok):
            self.tensor.append(self.done)
            yield from self.drain(self.done, 0)

    def softmax(self, q):
        works = tiles = outs = 0
        while True:
            w = yield from self.next_work(works)
            works += 1
            if not w:
                return
            nt, nq = w
            if q >= nq:
                continue
            for _ in range(nt):
                if not (yield from self.wait(self.sfull[q], tiles & 1)):
                    return
                tiles += 1
                for half in range(2):
                    yield
                    self.pfull[q][half].arrive()
            if self.output_warps:
                if outs > 0 and not (yield from self.wait(self.ofree[q], (outs - 1) & 1)):
                    return
                outs += 1
                self.rfull[q].arrive()
                continue
            if nt > 0:
                if not (yield from self.wait(self.ofull[q], outs & 1)):
                    return
                outs += 1
            self.finish(q)
            yield

    def finish(self, q):
        """The block's results: out of TMEM, or a cluster's partial ones over the ring."""
        if not self.cluster:
            self.ofree[q].arrive()
        elif any(self.filling.values()):
            raise Fault("partial results over a stage being filled")

    def output(self, warp):
        works = outs = stats = uses = 0
        while True:
            w = yield from self.next_work(works)
            works += 1
            if not w:
                return
            nt, nq = w
            for q in range(nq):
                if not (yield from self.wait(self.rfull[q], (stats >> q) & 1)):
                    return
                stats ^= 1 << q
                if nt > 0:
                    if not (yield from self.wait(self.ofull[q], (outs >> q) & 1)):
                        return
                    if self.cluster and nq == 2 and not (yield from self.wait(self.ofull[q ^ 1], (outs >> q) & 1)):
                        return
                    outs ^= 1 << q
                if self.cluster:
                    self.finish(q)
                    continue
                for half in range(2):
                    if uses > 0:
                        if warp == 0:
                            self.unstaged[half].arrive()
                        if not (yield from self.wait(self.unstaged[half], (uses - 1) & 1)):
                            return
                    yield
                    if half:
                        self.finish(q)
                    self.staged[half].arrive()
                    if warp == 0 and not (yield from self.wait(self.staged[half], uses & 1)):
                        return
                uses += 1

    # ------------------------------------------------------------ a run
    def run(self, most_steps=2_000_000):
        """Interleaves the roles until all have ended; returns whether one gave up."""
        rng = self.rng
        roles = [self.scheduler(), self.producer(), self.issuer()]
        roles += [self.softmax(q) for q in range(self.nq) for _ in range(self.warps)]
        roles += [self.output(w) for w in range(self.warps)] if self.output_warps else []
        speed = {id(r): rng.choice([1, 1, 2, 5]) for r in roles}
        copies, tensor = rng.choice([0.05, 0.3, 1, 3]), rng.choice([0.05, 0.3, 1, 3])
        for _ in range(most_steps):
            if not roles:
                break
            speeds = [speed[id(r)] for r in roles] + [copies if self.copies else 0, tensor if self.tensor else 0]
            k = rng.choices(range(len(speeds)), speeds)[0]
            if k < len(roles):
                try:
                    next(roles[k])
                except StopIteration:
                    roles.pop(k)
            elif k == len(roles):
                self.copies.pop(rng.randrange(len(self.copies)))()
            else:
                head = self.tensor.pop(0)
                if isinstance(head, Barrier):
                    head.arrive()
                while self.tensor and isinstance(self.tensor[0], Barrier):  # commits behind finished products
                    self.tensor.pop(0).arrive()
        if roles:
            raise Fault("does not end")
        if self.copies:
            raise Fault("exit with copies in flight")
        if self.tensor:
            raise Fault("exit with products or commits in flight")
        return self.abort


def trial(seed, give_up=None, mistakes=(), deep=False):
    """A random CTA; deep: one row tile and three stages, the ring's copies slow, many key tiles."""
    rng = random.Random(seed)
    row_tiles = 1 if deep else rng.choice([1, 1, 2])
    stages = 3 if deep else rng.choice([2, 3, 6]) if row_tiles == 1 else 4
    cluster = not deep and rng.random() < 0.3
    longest = 12 if deep else rng.choice([2, 5, 12])
    blocks = [(rng.randint(0 if cluster else 1, longest), rng.randint(1, row_tiles))
              for _ in range(1 if cluster else rng.randint(1, 6))]
    if give_up is None:
        give_up = rng.choice([0.0005, 0.002, 0.01, 0.05])
    return Cta(rng, row_tiles, stages, blocks, cluster, give_up, mistakes).run()

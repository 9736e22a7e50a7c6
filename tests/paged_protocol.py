"""The paged attention kernel's roles as coroutines: every barrier, and who may still read what.

A CTA of ``csrc/paged_attn.cuh`` has eleven roles at work (eight softmax warps, loads, MMA,
walk) and some forty barriers, whose waits tell a phase only from the one before it.  ``run``
plays them with the tensor core's queue and the copies in flight as two more actors, in an order
drawn from ``rng``, and raises ``Fault`` when

* a barrier gets more arrivals than it counts, a wait passes a phase early or can no longer
  tell that it is over, or nothing can go on;
* a score, probability or accumulator, a K, V or Q stage, a ring entry, a row statistic (``ml``)
  or a piece of the exchange area is read with another content than the one meant, or is
  written while a role has not read it yet;
* a copy (async proxy) writes to shared memory that ordinary stores have written, without a
  proxy fence in the storing warp in between.

``few_block(warp)`` is the block of sixteen ``ml`` entries that a warp uses when rows are few;
``fenced`` tells whether the warps fence the exchange area before they free it.

A segment is ``dict(kind=..., n=...)``: "few" (at most 16 rows), "single" (one row tile), "duo"
(two), "null" (no keys), of n key tiles.
"""

from __future__ import annotations

K_STAGES, V_STAGES, RING, READERS = 3, 2, 4, 9


class Fault(Exception):
    pass


class Bar:
    """An mbarrier: a count of arrivals, pending bytes, and waits by the parity of a phase."""

    def __init__(self, count, name):
        self.count, self.name = count, name
        self.pending, self.phase, self.bytes = count, 0, 0

    def _turn(self):
        if self.pending == 0 and self.bytes == 0:
            self.phase += 1
            self.pending = self.count

    def arrive(self, n=1, expect=0):
        if n > self.pending:
            raise Fault(f"{self.name}: too many arrivals")
        self.pending -= n
        self.bytes += expect
        self._turn()

    def landed(self, n):
        self.bytes -= n
        self._turn()

    def passes(self, phase):
        """Whether a wait for this phase returns now, by parity as the hardware does it."""
        yes = (self.phase & 1) != (phase & 1)
        if yes and self.phase <= phase:
            raise Fault(f"{self.name}: a wait for phase {phase} passes in phase {self.phase}")
        if not yes and self.phase > phase:
            raise Fault(f"{self.name}: a wait for phase {phase} misses it, now {self.phase}")
        return yes


class Shared:
    """A piece of shared memory with one content and the roles that still have to read it."""

    def __init__(self, name):
        self.name, self.content, self.readers = name, None, set()

    def write(self, content, readers):
        if self.readers:
            raise Fault(f"{self.name}: {content} over {self.content}, unread by {self.readers}")
        self.content, self.readers = content, set(readers)

    def read(self, content, reader):
        if self.content != content:
            raise Fault(f"{self.name}: {self.content} where {content} is meant")
        self.readers.discard(reader)


def run(segs, rng, few_block, fenced):
    bars = {}

    def bar(name, count, n):
        for i in range(n):
            bars[name, i] = Bar(count[i] if isinstance(count, tuple) else count, f"{name}({i})")

    bar("kfull", 1, K_STAGES)
    bar("kempty", READERS, K_STAGES)
    bar("vfull", 1, V_STAGES)
    bar("vempty", READERS, V_STAGES)
    bar("sfull", 1, 2)
    bar("phalf", 4, 2)
    bar("pfull", 4, 2)
    bar("odone", 1, 2)
    bar("ofree", (8, 4), 2)
    bar("qfull", 1, 2)
    bar("qfree", READERS, 2)
    bar("wfull", 1, RING)
    bar("wempty", 10, RING)
    bar("xch", 4, 1)
    bar("few", 8, 1)
    k_tile, v_tile, q_tile = [None] * K_STAGES, [None] * V_STAGES, [None] * 2
    score, probs, acc, products = [None] * 2, [{}, {}], [None] * 2, [0, 0]
    ml = [Shared(f"ml[{16 * b}]") for b in range(8)]
    area = [Shared(f"exchange area of warp {w}") for w in range(8)]
    unfenced = set()               # warps whose stores to the exchange area have no fence yet
    ring = [None] * RING
    copies = []                    # in flight, in any order
    queue = []                     # the tensor core's, in order

    def wait(name, i, phase):
        return bars[name, i], phase

    def take(i):
        yield wait("wfull", i % RING, i // RING)
        seg = ring[i % RING]
        if seg is not None and seg["i"] != i:
            raise Fault("ring entry")
        bars["wempty", i % RING].arrive()
        return seg

    def walk():
        turn, uses = 0, [0, 0]
        for i, s in enumerate(segs + [None]):
            if i >= RING:
                yield wait("wempty", i % RING, i // RING - 1)
            if s is not None:
                both = s["kind"] in ("few", "duo")
                s = dict(s, i=i, buf=turn, use=[None, None])
                if s["kind"] != "null":
                    for b in range(2):
                        if both or b == turn:
                            s["use"][b] = uses[b]
                            uses[b] += 1
                    if not both:
                        turn ^= 1
            ring[i % RING] = s
            bars["wfull", i % RING].arrive()
            yield None

    def loads():
        kt = i = 0
        while True:
            seg = yield from take(i)
            i += 1
            if seg is None:
                return
            if seg["kind"] == "null":
                continue
            for b in range(2):
                use = seg["use"][b]
                if use is None:
                    continue
                if use > 0:
                    yield wait("qfree", b, use - 1)
                if seg["kind"] == "few":
                    bars["qfull", b].arrive()
                    q_tile[b] = ("area", seg["i"])
                    continue
                q_tile[b] = None
                bars["qfull", b].arrive(1, 1)
                copies.append(("q", b, (seg["i"], b if seg["kind"] == "duo" else 0)))
            for _ in range(seg["n"]):
                ks, vs = kt % K_STAGES, kt % V_STAGES
                if kt >= K_STAGES:
                    yield wait("kempty", ks, kt // K_STAGES - 1)
                k_tile[ks] = None
                bars["kfull", ks].arrive(1, 1)
                copies.append(("k", ks, kt))
                yield None
                if kt >= V_STAGES:
                    yield wait("vempty", vs, kt // V_STAGES - 1)
                v_tile[vs] = None
                bars["vfull", vs].arrive(1, 1)
                copies.append(("v", vs, kt))
                yield None
                kt += 1

    def mma():
        kt = i = 0
        uses_p, uses_o = [0, 0], [0, 0]

        def commit_all(name, j):
            bars[name, j].arrive(READERS - 1)
            queue.append(("commit", bars[name, j]))

        def qk(seg, j):
            duo = seg["kind"] == "duo"
            h, k = j & 1, kt + (j >> duo)
            st, qb = k % K_STAGES, h if duo else seg["buf"]
            if j < 2 and (duo or j == 0):
                yield wait("qfull", qb, seg["use"][qb])
            yield wait("kfull", st, k // K_STAGES)
            queue.append(("qk", h, st, k, qb, (seg["i"], h if duo else 0), (seg["i"], j >> duo)))
            queue.append(("commit", bars["sfull", h]))
            if not duo or h == 1:
                commit_all("kempty", st)
            if j + 1 + duo >= seg["n"] << duo:
                commit_all("qfree", qb)

        def pv(seg, j):
            duo = seg["kind"] == "duo"
            h, k = j & 1, kt + (j >> duo)
            st, use = k % V_STAGES, uses_p[h]
            uses_p[h] += 1
            yield wait("vfull", st, k // V_STAGES)
            if not duo or h == 0:              # clears the rows behind the last key
                if v_tile[st] != (k, "landed"):
                    raise Fault("V stage to be cleared")
                v_tile[st] = (k, "cleared")
            if j < 2:
                if uses_o[h] > 0:
                    yield wait("ofree", h, uses_o[h] - 1)
                uses_o[h] += 1
            yield wait("phalf", h, use)
            products[h] += 1
            queue.append(("pv", h, st, k, (seg["i"], j >> duo), 0))
            yield wait("pfull", h, use)
            products[h] += 1
            queue.append(("pv", h, st, k, (seg["i"], j >> duo), 1))
            if not duo or h == 1:
                commit_all("vempty", st)
            if j + 2 >= seg["n"] << duo:
                queue.append(("commit", bars["odone", h]))

        while True:
            seg = yield from take(i)
            i += 1
            if seg is None:
                return
            if seg["kind"] == "null":
                continue
            if seg["kind"] == "few":           # sees every phase, and holds up the next
                for b in range(2):
                    yield wait("qfull", b, seg["use"][b])
                    bars["qfree", b].arrive()
                for _ in range(seg["n"]):
                    yield wait("kfull", kt % K_STAGES, kt // K_STAGES)
                    bars["kempty", kt % K_STAGES].arrive()
                    yield wait("vfull", kt % V_STAGES, kt // V_STAGES)
                    bars["vempty", kt % V_STAGES].arrive()
                    kt += 1
                continue
            steps = seg["n"] << (seg["kind"] == "duo")
            for j in range(min(2, steps)):
                yield from qk(seg, j)
            for j in range(steps):
                yield from pv(seg, j)
                yield None
                if j + 2 < steps:
                    yield from qk(seg, j + 2)
            kt += seg["n"]

    def softmax(w):
        hd, quad = w >> 2, w & 3
        steps = joins = kt = fews = 0
        uses_o = [0, 0]
        i = -1
        while True:
            i += 1
            yield wait("wfull", i % RING, i // RING)
            seg = ring[i % RING]
            if seg is None:
                return
            if seg["i"] != i:
                raise Fault("ring entry")
            kind, n = seg["kind"], seg["n"]
            if kind == "few":
                bars["wempty", i % RING].arrive()
                for _ in range(n):
                    yield wait("kfull", kt % K_STAGES, kt // K_STAGES)
                    if k_tile[kt % K_STAGES] != kt:
                        raise Fault("K stage, few rows")
                    yield None
                    if k_tile[kt % K_STAGES] != kt:
                        raise Fault("K stage, few rows, late")
                    bars["kempty", kt % K_STAGES].arrive()
                    yield wait("vfull", kt % V_STAGES, kt // V_STAGES)
                    if v_tile[kt % V_STAGES] != (kt, "landed"):
                        raise Fault("V stage, few rows")
                    yield None
                    if v_tile[kt % V_STAGES] != (kt, "landed"):
                        raise Fault("V stage, few rows, late")
                    bars["vempty", kt % V_STAGES].arrive()
                    kt += 1
                for b in range(2):
                    yield wait("qfull", b, seg["use"][b])
                if hd == 1 and uses_o[1] > 0:
                    yield wait("ofree", 1, uses_o[1] - 1)
                if q_tile != [("area", i)] * 2:
                    raise Fault("exchange area not free")
                area[w].write(i, range(8))
                unfenced.add(w)
                ml[few_block(w)].write(("few", i, w), range(8))
                yield None
                bars["few", 0].arrive()
                yield wait("few", 0, fews)
                fews += 1
                for v in range(8):
                    area[v].read(i, w)
                    ml[few_block(v)].read(("few", i, v), w)
                    yield None
                if fenced:
                    unfenced.discard(w)
                for b in range(2):
                    bars["qfree", b].arrive()
                continue
            duo, none = kind == "duo", kind == "null"
            two = kind == "single" and n > 1
            if not none:
                started = False
                for t in range(0 if duo else hd, n, 1 if duo else 2):
                    yield wait("sfull", hd, steps)
                    steps += 1
                    if score[hd] != (i, t):
                        raise Fault("scores")
                    yield None
                    if started and rng.random() < 0.3:          # rescales the accumulator
                        for _ in range(2):
                            if products[hd]:
                                raise Fault("rescale while a product is under way")
                            yield None
                    started = True
                    if score[hd] != (i, t):
                        raise Fault("scores, late")
                    probs[hd][w, 0] = (i, t)
                    bars["phalf", hd].arrive()
                    yield None
                    probs[hd][w, 1] = (i, t)
                    bars["pfull", hd].arrive()
                kt += n
            use = list(uses_o)
            if not none:
                uses_o[0] += 1
                uses_o[1] += duo or two
            if ring[i % RING] is None or ring[i % RING]["i"] != i:
                raise Fault("ring entry read again")
            bars["wempty", i % RING].arrive()
            if none:
                continue
            if not duo and hd == 1:
                if two:
                    if use[1] > 0:
                        yield wait("ofree", 1, use[1] - 1)
                    for b in (2 * quad, 2 * quad + 1):
                        ml[b].write(("two", i), [quad])
                    yield None
                    bars["xch", 0].arrive()
                    yield wait("odone", 1, use[1])
                yield wait("odone", 0, use[0])
                bars["ofree", 0].arrive()
                continue
            if two:
                yield wait("xch", 0, joins)
                joins += 1
            yield wait("odone", 0, use[0])
            if hd == 1:
                bars["ofree", 0].arrive()
                yield wait("odone", 1, use[1])
            if two:
                yield wait("odone", 1, use[1])
                yield None                                      # the warps part here
                for b in (2 * quad, 2 * quad + 1):
                    ml[b].read(("two", i), quad)
            mine = [hd] if duo else [0, 1] if two else [0]
            for _ in range(2):
                for h in mine:
                    last = n - 1 if duo or (n - 1) % 2 == h else n - 2
                    if acc[h] != (i, last) or products[h]:
                        raise Fault("accumulator")
                yield None
            bars["ofree", hd].arrive()
            if two:
                bars["ofree", 1].arrive()

    def land(kind, st, value):
        if kind == "k":
            k_tile[st] = value
            bars["kfull", st].landed(1)
        elif kind == "v":
            v_tile[st] = (value, "landed")
            bars["vfull", st].landed(1)
        else:
            if unfenced:
                raise Fault(f"a copy over unfenced stores of warps {unfenced}")
            if any(a.readers for a in area):
                raise Fault("a copy over an exchange area in use")
            q_tile[st] = value
            bars["qfull", st].landed(1)

    def execute(op):
        if op[0] == "commit":
            op[1].arrive()
        elif op[0] == "qk":
            _, h, st, k, qb, rows, step = op
            if k_tile[st] != k or q_tile[qb] != rows:
                raise Fault("operands of a score product")
            score[h], probs[h] = step, {}
        else:
            _, h, st, k, step, half = op
            if v_tile[st] != (k, "cleared"):
                raise Fault("V stage of a product")
            if [x for (_, part), x in probs[h].items() if part == half] != [step] * 4:
                raise Fault("probabilities of a product")
            acc[h] = step
            products[h] -= 1

    roles = {"walk": walk(), "loads": loads(), "mma": mma()}
    roles.update({f"softmax {w}": softmax(w) for w in range(8)})
    state = dict.fromkeys(roles)
    # some roles are slow, some fast
    pace = {r: rng.choice([1, 1, 1, 5, 25]) for r in roles}
    pace["copies"], pace["queue"] = rng.choice([1, 5, 25]), rng.choice([1, 5, 25])
    while state or copies or queue:
        ready = [r for r, at in state.items() if at is None or at[0].passes(at[1])]
        ready += ["copies"] * bool(copies) + ["queue"] * bool(queue)
        if not ready:
            raise Fault("nothing goes on: " + ", ".join(f"{r} at {at[0].name} phase {at[1]}"
                                                        for r, at in state.items()))
        r = rng.choices(ready, [pace[x] for x in ready])[0]
        if r == "copies":
            land(*copies.pop(rng.randrange(len(copies))))
        elif r == "queue":
            execute(queue.pop(0))
        else:
            try:
                state[r] = next(roles[r])
            except StopIteration:
                del state[r]


KINDS = (["few"], ["single"], ["duo"], ["few", "single"], ["few", "duo"], ["single", "duo"],
         ["few", "single", "duo"], ["few", "single", "duo", "null"])


def random_segments(rng):
    kinds, most = rng.choice(KINDS), rng.choice([1, 2, 4, 9])
    return [dict(kind=rng.choice(kinds), n=rng.randint(1, most)) for _ in range(rng.randint(1, 14))]

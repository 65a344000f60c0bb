"""Write nt_loop.inc: the K loops of the large tiles of nt_loop.h as GCN assembly
text for gfx950.

The C++ part sets up addresses and runs the epilogue; the loop is written
instruction by instruction, because the compiler neither keeps sums, fragments
and prefetches of a 128 x 64 wavefront tile within 256 registers nor keeps the
products between the reads that they hide.

A loop sums a block tile of 16 MT WM x 16 NT WN over steps of 128 bytes of K.
Two stages lie in LDS, a power of two apart; a stage is A's panel, B's panel
(rows of 128 bytes, 16-byte chunk c of row r in slot c ^ ((r / 2) % 8)) and,
behind both stages, the scales of the stage's rows (4 bytes each).

A step's MT x NT products are taken in four quarters, two halves of A by two of
B, in the order (0, x) (0, y) (1, y) (1, x), with x = 0, y = 1 in stage 0 and
the reverse in stage 1: each quarter but the first of a step changes one half
only, and what it needs is read during the quarter before it, over the step's
end too.  The loads of the step after next go to the stage whose last reads all
wavefronts have made by the end of the third quarter, where the step's only
barrier is.

Kinds:
  e8m0   8-bit products, power-of-two scales applied by the instruction
  f32u   8-bit products summed from zero, then added times the product of A's
         row's scale and the one scale of the wavefront's B rows
  f32n   the same with a scale for each of B's rows
  pair   numbers as pairs of halfs (64 bytes hi, 64 bytes lo), three products
Products that are scaled afterwards lie in a ring of four results, and each is
added after three more have been issued, when it has arrived.

Run as a script to rewrite nt_loop.inc; a test checks that the committed file
is what this writes.
"""

from __future__ import annotations

import os

OUT = os.path.join(os.path.dirname(os.path.abspath(__file__)), "nt_loop.inc")


class Loop:
    """One loop's text.  Registers: v[0:..] the sums, (j MT + i) 4; then the
    fragments of A and B, the ring of results, A's and B's scales."""

    def __init__(self, kind, mt, nt, wm, wn):
        self.kind, self.mt, self.nt = kind, mt, nt
        self.hm, self.hn = mt // 2, nt // 2
        self.waves = wm * wn
        self.bm, self.bn = 16 * mt * wm, 16 * nt * wn
        self.la, self.lb = self.bm // 8 // self.waves, self.bn // 8 // self.waves
        self.stride = 1 << (128 * (self.bm + self.bn) - 1).bit_length()
        self.scaled = kind != "pair"
        self.after = kind in ("f32u", "f32n")
        self.scale_waves = (self.bm + self.bn) // 64
        self.scale_stage = 256 * self.waves * self.scale_loads
        self.lines = []
        at = 4 * mt * nt
        # as many slots for A as registers allow: half of MT, each reused when its products are issued, or all
        self.slots = mt if mt <= 4 else mt // 2
        self.a0, at = at, at + 8 * self.slots
        self.b0, at = at, at + 8 * nt
        self.t0, at = at, at + (16 if self.after else 0)
        self.sm0, at = at, at + (mt if self.scaled else 0)
        self.sn0, at = at, at + {"e8m0": nt, "f32u": 2, "f32n": 4 * nt, "pair": 0}[kind]
        self.registers = at
        self.reads = []    # LDS reads under way, oldest first: the registers' names
        self.pending = []  # products not yet added: (result, j, i), oldest first

    @property
    def scale_loads(self):
        """Loads of 64 scales a wavefront."""
        return -(-((self.bm + self.bn) // 64) // self.waves) if self.scaled else 0

    # -- text

    def emit(self, text):
        self.lines.append(text)

    def acc(self, j, i):
        at = 4 * (j * self.mt + i)
        return f"v[{at}:{at + 3}]"

    def fa(self, i, part=None):
        return self._frag(self.a0 + 8 * (i % self.slots), part)

    def fb(self, j, part=None):
        return self._frag(self.b0 + 8 * j, part)

    @staticmethod
    def _frag(at, part):
        if part is None:
            return f"v[{at}:{at + 7}]"
        return f"v[{at + 4 * part}:{at + 4 * part + 3}]"

    def sm(self, i):
        return f"v{self.sm0 + i}"

    def sn(self, j, r=0):
        return f"v{self.sn0 + (4 * j + r if self.kind == 'f32n' else j)}"

    # -- LDS reads; `name` says what arrives with them

    def read(self, text, name):
        self.emit(text)
        self.reads.append(name)

    def need(self, names):
        """Wait until these have arrived."""
        last = max((k for k, n in enumerate(self.reads) if n in names), default=-1)
        if last >= 0:
            self.emit(f"s_waitcnt lgkmcnt({min(len(self.reads) - 1 - last, 15)})")
            self.reads = self.reads[last + 1:]

    # The scales of results still in the ring must stay until these are added, which
    # is after the third product of the next quarter: from then on new ones may come.
    SETTLED = 2

    def a_reads(self, i):
        yield lambda: self.read(f"ds_read_b128 {self.fa(i, 0)}, %[aLo] offset:{2048 * i}", ("a", i))
        yield lambda: self.read(f"ds_read_b128 {self.fa(i, 1)}, %[aHi] offset:{2048 * i}", ("a", i))
        if self.scaled:
            yield lambda: self.read(f"ds_read_b32 {self.sm(i)}, %[aS] offset:{64 * i}", ("sa", i))

    def b_reads(self, j):
        yield lambda: self.read(f"ds_read_b128 {self.fb(j, 0)}, %[bLo] offset:{2048 * j}", ("b", j))
        yield lambda: self.read(f"ds_read_b128 {self.fb(j, 1)}, %[bHi] offset:{2048 * j}", ("b", j))
        if self.kind == "e8m0":
            yield lambda: self.read(f"ds_read_b32 {self.sn(j)}, %[bS] offset:{64 * j}", ("sb", j))
        elif self.kind == "f32n":
            at = self.sn0 + 4 * j
            yield lambda: self.read(f"ds_read_b128 v[{at}:{at + 3}], %[bS] offset:{64 * j}", ("sb", j))

    def uniform_read(self, stage):
        """The wavefront's one scale of B, of the step in `stage`."""
        if self.kind == "f32u":
            yield lambda: self.read(f"ds_read_b32 {self.sn(stage)}, %[bS]", ("su", stage))

    # -- loads to LDS

    def dma(self, stage, loads):
        """Loads number `loads` (A's, B's, then the scales') of a step into `stage`."""
        for n in loads:
            if n < self.la + self.lb:
                side, k, base = ("A", n, 0) if n < self.la else ("B", n - self.la, 128 * self.bm)
                lane = f"%[{side.lower()}{'Odd' if k % 2 else 'Even'}]"
                rs = "s[60:63]" if side == "A" else "s[64:67]"

                def one(side=side, k=k, base=base, lane=lane, rs=rs):
                    self.emit(f"s_add_u32 m0, %[lds{side}], {stage * self.stride + base + 1024 * k}")
                    self.emit("s_nop 0")
                    self.emit(f"buffer_load_dwordx4 {lane}, {rs}, %[o{side}{k}] offen lds")
                yield one
            elif n < self.loads:
                k = n - self.la - self.lb

                def one(k=k):
                    size = "ubyte" if self.kind == "e8m0" else "dword"
                    at = 2 * self.stride + stage * self.scale_stage + 256 * self.waves * k
                    self.emit(f"s_add_u32 m0, %[ldsS], {at}")
                    self.emit("s_nop 0")
                    self.emit(f"global_load_lds_{size} %[gS{k}], s[68:69]")
                yield one
            else:
                yield self.advance

    @property
    def loads(self):
        return self.la + self.lb + self.scale_loads

    def advance(self):
        """On to the next step's."""
        for lo in (60, 64):
            self.emit(f"s_add_u32 s{lo}, s{lo}, 128")
            self.emit(f"s_addc_u32 s{lo + 1}, s{lo + 1}, 0")
            self.emit(f"s_sub_u32 s{lo + 2}, s{lo + 2}, 128")
        if self.scaled:
            self.emit("s_add_u32 s68, s68, s70")
            self.emit("s_addc_u32 s69, s69, s71")

    # -- products

    def add(self, entry):
        """A result that has arrived into its sum, times its scales."""
        t, j, i = entry
        at = 4 * (j * self.mt + i)
        if self.kind == "f32n":
            self.need([("sa", i), ("sb", j)])
            for r in range(4):
                self.emit(f"v_mul_f32 v{t + r}, v{t + r}, {self.sm(i)}")
            for r in range(4):
                self.emit(f"v_fmac_f32 v{at + r}, v{t + r}, {self.sn(j, r)}")
        else:
            for r in range(4):
                self.emit(f"v_fmac_f32 v{at + r}, v{t + r}, {self.sm(i)}")

    def masks(self, names):
        """Zero what lies past K's end of fragments that have arrived."""
        for side, n in names:
            at = (self.a0 + 8 * (n % self.slots)) if side == "a" else self.b0 + 8 * n
            for r in range(8):
                self.emit(f"v_and_b32 v{at + r}, v{at + r}, %[mask{'Lo' if r < 4 else 'Hi'}{r % 4}]")
        if names:
            self.emit("s_nop 1")

    def quarter(self, ih, jh, stage, side, masked=()):
        """The products of halves ih of A and jh of B; `side`: what to issue
        between them, entries (first, f): f after product number `first` or later."""
        side = list(side)
        group = 2 if self.kind == "pair" else 1
        order = []
        for i0 in range(0, self.hm, group):
            for term in range(3 if self.kind == "pair" else 1):
                for i in range(i0, min(i0 + group, self.hm)):
                    for j in range(self.hn):
                        order.append((ih * self.hm + i, jh * self.hn + j, term))
        # evenly over the products, none before its time
        total = len(order)
        fresh = set(masked)
        for n, (i, j, term) in enumerate(order):
            self.need([("a", i), ("b", j)] + ([("sa", i), ("sb", j)] if self.kind == "e8m0" else []))
            now = [x for x in (("a", i), ("b", j)) if x in fresh]
            if now:
                fresh -= set(now)
                self.masks(now)
            a, b = self.fa(i), self.fb(j)
            if self.kind == "e8m0":
                self.emit(f"v_mfma_scale_f32_16x16x128_f8f6f4 {self.acc(j, i)}, {b}, {a}, {self.acc(j, i)}, "
                          f"{self.sn(j)}, {self.sm(i)} op_sel_hi:[0,0,0]")
            elif self.kind == "pair":
                self.emit(f"v_mfma_f32_16x16x32_f16 {self.acc(j, i)}, {self.fb(j, int(term == 2))}, "
                          f"{self.fa(i, int(term == 1))}, {self.acc(j, i)}")
            else:
                t = self.t0 + 4 * (self.count % 4)
                self.count += 1
                self.emit(f"v_mfma_f32_16x16x128_f8f6f4 v[{t}:{t + 3}], {b}, {a}, 0")
                if self.kind == "f32u" and (ih, jh) in ((0, stage), (1, 1 - stage)) and j == jh * self.hn:
                    # this half's first quarter: A's scale becomes the product of both
                    self.need([("sa", i), ("su", stage)])
                    self.emit(f"v_mul_f32 {self.sm(i)}, {self.sm(i)}, {self.sn(stage)}")
                self.pending.append((t, j, i))
                if len(self.pending) > 3:
                    self.add(self.pending.pop(0))
            left = total - n - 1
            due = [s for s in side if s[0] <= n]
            later = len(side) - len(due)
            take = -(-len(due) // max(1, left - (later > 0) + 1)) if left else len(side)
            for s in (due if left else list(side))[:take]:
                side.remove(s)
                s[1]()
        assert not side

    def meet(self):
        self.emit("s_waitcnt vmcnt(0) lgkmcnt(0)")
        self.reads = []
        self.emit("s_barrier")

    def turn(self, stage):
        """The reads' places move to `stage`."""
        sign = 1 if stage else -1
        for n in ("aLo", "aHi", "bLo", "bHi"):
            self.emit(f"v_add_u32 %[{n}], {sign * self.stride}, %[{n}]")
        if self.scaled:
            for n in ("aS", "bS"):
                self.emit(f"v_add_u32 %[{n}], {sign * self.scale_stage}, %[{n}]")

    def step(self, x, still, masked=False):
        """A step out of stage x, whose first halves have been read; still: how
        many steps follow, 2 for more."""
        y = 1 - x
        split = (self.loads * 5 + 8) // 9
        halves = lambda side, h: [(side, h * n + k) for n in [self.hm if side == "a" else self.hn] for k in range(n)]  # noqa: E731
        m = lambda names: names if masked else ()  # noqa: E731
        per = self.hn * (3 if self.kind == "pair" else 1)  # products a fragment of A has in a quarter
        group = 2 if self.kind == "pair" else 1

        side = self.b_side(y)
        if self.slots == self.mt:  # room beside the first half
            side += [(self.SETTLED if self.after else 0, f) for i in range(self.hm) for f in self.a_reads(self.hm + i)]
        if still > 0:
            side = self.merged(side, [(0, f) for f in self.dma(y, range(split, self.loads + 1))])
        self.quarter(0, x, x, side, m(halves("a", 0) + halves("b", x)))

        side = []
        if self.slots < self.mt:
            for i in range(self.hm):
                done = per * (i // group * group + group) - 1
                side += [(done, f) for f in self.a_reads(self.hm + i)]
        self.quarter(0, y, x, side, m(halves("b", y)))
        self.quarter(1, y, x, [], m(halves("a", 1)))
        side = []
        if still > 0:
            self.meet()
            self.turn(y)
            side += self.b_side(y)
            side += [(0, f) for f in self.uniform_read(y)]
            for i in range(self.hm):
                done = 0 if self.slots == self.mt else per * (i // group * group + group) - 1
                side += [(done, f) for f in self.a_reads(i)]
        if still > 1:
            side = self.merged(side, [(0, f) for f in self.dma(x, range(split))])
        self.quarter(1, x, x, side)

    def b_side(self, half):
        """The reads of a half of B, as a quarter's side entries."""
        late = self.SETTLED if self.kind == "f32n" else 0
        reads = [list(self.b_reads(half * self.hn + j)) for j in range(self.hn)]
        return [(0, f) for r in reads for f in r[:2]] + [(late, f) for r in reads for f in r[2:]]

    @staticmethod
    def merged(reads, loads):
        """Loads evenly among the reads."""
        out, n = [], len(loads)
        for k, entry in enumerate(reads):
            out.append(entry)
            while loads and (n - len(loads)) * len(reads) <= k * n:
                out.append(loads.pop(0))
        return out + loads

    def start(self, x):
        """The first step into stage x."""
        for f in self.dma(x, range(self.loads + 1)):
            f()
        for n in range(4 * self.mt * self.nt):
            self.emit(f"v_mov_b32 v{n}, 0")
        for n in range(self.t0, self.registers):
            self.emit(f"v_mov_b32 v{n}, 0")
        self.meet()
        if x == 1:
            self.turn(1)
        for f in self.uniform_read(x):
            f()
        for i in range(self.hm):
            for f in self.a_reads(i):
                f()
        for j in range(self.hn):
            for f in self.b_reads(x * self.hn + j):
                f()
        self.emit("s_waitcnt lgkmcnt(0)")
        self.reads = []

    def first_part(self, x):
        for f in self.dma(x, range((self.loads * 5 + 8) // 9)):
            f()

    def text(self):
        """The whole loop; %[steps] >= 1, the last step in stage 1."""
        # what is under way and pending where a step begins: as the step before leaves it
        probe = Loop(self.kind, self.mt, self.nt, self.waves, 1)
        probe.__dict__.update({k: v for k, v in self.__dict__.items() if k not in ("lines", "reads", "pending")})
        probe.lines, probe.reads, probe.pending, probe.count = [], [], [], 0
        begin = {}
        for x in (0, 1, 0, 1, 0, 1):
            begin[x] = (list(probe.reads), list(probe.pending), probe.count % 4)
            probe.step(x, 2)
        assert begin[0] == (probe.reads, probe.pending, probe.count % 4)

        def enter(x):
            reads, pending, count = begin[x]
            self.reads, self.pending, self.count = list(reads), list(pending), count

        def check(x):
            assert (self.reads, self.pending, self.count % 4) == begin[x], (x, self.reads, begin[x])

        self.count = 0
        self.emit("s_bitcmp1_b32 %[steps], 0")
        self.emit("s_cbranch_scc1 .Lnt_odd_%=")
        self.start(0)
        self.emit("s_branch .Lnt_even_%=")
        self.emit(".Lnt_odd_%=:")
        self.start(1)
        self.emit("s_cmp_eq_u32 %[steps], 1")
        self.emit("s_cbranch_scc1 .Lnt_last_%=")
        self.first_part(0)
        enter(1)
        self.step(1, 2)
        check(0)
        self.emit("s_branch .Lnt_pairs_%=")
        self.emit(".Lnt_even_%=:")
        self.first_part(1)
        self.emit(".Lnt_pairs_%=:")
        self.emit("s_sub_u32 %[steps], %[steps], 2")
        self.emit("s_lshr_b32 %[steps], %[steps], 1")
        self.emit("s_cmp_eq_u32 %[steps], 0")
        self.emit("s_cbranch_scc1 .Lnt_next_%=")
        self.emit(".Lnt_loop_%=:")
        enter(0)
        self.step(0, 2)
        check(1)
        self.step(1, 2)
        check(0)
        self.emit("s_sub_u32 %[steps], %[steps], 1")
        self.emit("s_cmp_lg_u32 %[steps], 0")
        self.emit("s_cbranch_scc1 .Lnt_loop_%=")
        self.emit(".Lnt_next_%=:")
        enter(0)
        self.step(0, 1)
        check(1)
        self.emit(".Lnt_last_%=:")
        if self.scaled:
            self.emit("s_cmp_lg_u32 %[partial], 0")
            self.emit("s_cbranch_scc1 .Lnt_masked_%=")
        enter(1)
        self.step(1, 0)
        self.drain()
        if self.scaled:
            self.emit("s_branch .Lnt_end_%=")
            self.emit(".Lnt_masked_%=:")
            enter(1)
            self.step(1, 0, masked=True)
            self.drain()
            self.emit(".Lnt_end_%=:")
        return self.lines

    def drain(self):
        self.emit("s_waitcnt lgkmcnt(0)")
        self.reads = []
        self.emit("s_nop 15")
        self.emit("s_nop 7")
        for p in self.pending:
            self.add(p)
        self.pending = []

    def name(self):
        return f"{self.kind}_{self.bm}x{self.bn}"


LOOPS = [
    ("e8m0", 8, 4, 2, 4), ("f32u", 8, 4, 2, 4), ("f32n", 8, 4, 2, 4), ("pair", 8, 4, 2, 4),
]


def generate() -> str:
    out = ["// Generated by gen_nt_loop.py (the K loops of nt_loop.h); do not edit."]
    for args in LOOPS:
        loop = Loop(*args)
        loop.count = 0
        name = loop.name()
        text = loop.text()
        out.append(f"#define NT_LOOP_{name} \\")
        out += [f'  "{line}\\n" \\' for line in text]
        out.append('  ""')
        spare = range(4 * loop.mt * loop.nt, loop.registers)
        out.append(f"#define NT_CLOBBERS_{name} " + ", ".join(f'"v{n}"' for n in spare))
    return "\n".join(out) + "\n"


if __name__ == "__main__":
    with open(OUT, "w") as f:
        f.write(generate())

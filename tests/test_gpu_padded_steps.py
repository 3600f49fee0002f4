"""Steps on the rows that the batch tables give, padding included: a captured
step runs on a fixed number of rows, idle and finished sequences leave some of
them empty, and the calls of the path skip those without a status bit and
leave what they would write as it was."""
import pytest
import torch

from deepseek_v4_compressed_gb300 import binding as B

pytestmark = pytest.mark.gpu

S, ROWS, H, HI, K, CTX = 6, 12, 8, 16, 64, 2048


def i32(*shape, fill=0):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


class Step:
    """A layer's step over ROWS rows: tables, the two compressors, the window
    rows, the indexer and the attention (V4 rows with quantised output, or the
    576 geometry)."""

    def __init__(self, v4, fp4, lengths, seed=0, plan_ctx=CTX):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.v4, self.idx_kind = v4, B.CACHE_IDX_FP4 if fp4 else B.CACHE_IDX
        self.main_kind, d = (B.CACHE_V4, 512) if v4 else (B.CACHE_MLA, 576)
        self.status = i32(1)
        self.computed, self.new = i32(S), i32(S)
        self.meta = dict(offsets=i32(S + 1), ctx_len=i32(S), positions=i32(ROWS), seqs=i32(ROWS), row_ctx=i32(ROWS))
        self.groups = []
        for ratio, window in ((1, 128), (4, 0)):
            pages, width = S * 12, CTX // ratio // 64
            owned, at = torch.full((S, width), -1, dtype=torch.int32), 0
            perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed + ratio)).int()
            for s, c in enumerate(lengths):
                for j in range(max(0, c - window + 1) // 64 if window else 0, -(-(c // ratio) // 64)):
                    owned[s, j] = perm[at]
                    at += 1
            ring = torch.full((pages,), -1, dtype=torch.int32)
            ring[:pages - at] = perm[at:]
            self.groups.append(B.TableGroup(ratio=ratio, window=window, num_pages=pages, owned=owned.cuda(), table=i32(S, width), ring=ring.cuda(),
                                            pool_in=torch.tensor([0, pages - at], device="cuda"), pool_out=torch.zeros(2, dtype=torch.int64, device="cuda"),
                                            slots=torch.zeros(ROWS, dtype=torch.int64, device="cuda")))
        self.tables = B.BatchTables(self.groups, num_seqs=S, max_tokens=ROWS, status=self.status, **self.meta)
        self.swa = torch.zeros(S * 12 * (B.V4_PAGE_BYTES if v4 else B.SWA_PAGE_BYTES), dtype=torch.uint8, device="cuda")
        self.comp = torch.zeros(S * 12 * B.PAGE_BYTES[self.main_kind], dtype=torch.uint8, device="cuda")
        self.idx = torch.zeros(S * 12 * B.PAGE_BYTES[self.idx_kind], dtype=torch.uint8, device="cuda")
        self.states = [rand(S, 8, 4 * n) for n in (d, 128)]
        self.inputs = [dict(kv_score=rand(ROWS, 4 * n).bfloat16(), ape=rand(4, 2 * n), rms_weight=rand(n)) for n in (d, 128)]
        self.cs = B.rope_table(CTX).cuda()
        self.rows = rand(ROWS, 512) / 512 ** 0.5
        self.qi = rand(ROWS, HI, 128).to(torch.float8_e4m3fn).view(torch.uint8)
        self.w = torch.rand((ROWS, HI), generator=g, device="cuda")
        self.q = rand(ROWS, H, 512 if v4 else 576).bfloat16()
        self.plan = B.Plan(B.C4A, H, ROWS, K, plan_ctx, idx_heads=HI, idx_format=B.IDX_FP4 if fp4 else B.IDX_FP8, kv_layout=B.KV_V4 if v4 else B.KV_576)
        self.ws = self.plan.workspace()
        self.out = dict(idx=i32(ROWS, K), len=i32(ROWS), out=torch.zeros((ROWS, H, 512), dtype=torch.bfloat16, device="cuda"), lse=torch.zeros((ROWS, H), device="cuda"),
                        codes=torch.zeros((ROWS, H, 512), dtype=torch.uint8, device="cuda"), scales=torch.zeros((ROWS, H, 4), device="cuda"))
        # the entries and window rows cached before, through the tables of an idle step
        self.computed.copy_(torch.tensor(lengths))
        self.tables.build(self.computed, self.new)
        for s, c in enumerate(lengths):
            for kind, cache, table, n, width in ((self.main_kind, self.comp, 1, c // 4, d), (self.idx_kind, self.idx, 1, c // 4, 128), (B.CACHE_V4, self.swa, 0, c, 512)):
                lo = max(0, c - 127) // 64 * 64 if table == 0 else 0
                if n > lo and (v4 or table):
                    B.cache_insert_rows(kind, rand(n - lo, width) / width ** 0.5, i32(n - lo, fill=s), torch.arange(lo, n, dtype=torch.int32, device="cuda"), cache, self.groups[table].table,
                                        status=self.status)
        if not v4:
            self.swa.copy_((rand(self.swa.numel() // 2) / 24).bfloat16().view(torch.uint8))
        assert B.read_device_status(self.status)[1] == 0

    def clear(self):
        """Outputs that no call writes."""
        for k, t in self.out.items():
            t.copy_(torch.full_like(t.float(), 77.0).to(t.dtype))

    def tables_step(self):
        self.tables.build(self.computed, self.new)

    def path(self, n, seqs, positions, row_ctx, one_token=True):
        """The path on the first n rows; the indexer and attention on all, by
        the given rows' sequences and lengths."""
        args = [dict(kind=kind, ratio=4, kv_score=x["kv_score"][:n], positions=positions[:n], seqs=seqs[:n], ape=x["ape"], rms_weight=x["rms_weight"], rms_eps=1e-6,
                     cos_sin=self.cs, state=state, cache=cache, block_table=self.groups[1].table, num_seqs=S, status=self.status)
                for kind, x, state, cache in zip((self.main_kind, self.idx_kind), self.inputs, self.states, (self.comp, self.idx))]
        if one_token:
            B.compress_insert_pair(*args)
        else:
            for a in args:
                B.compress_insert(one_token_per_seq=False, **a)
        if self.v4:
            B.cache_insert_rows(B.CACHE_V4, self.rows[:n], seqs[:n], positions[:n], self.swa, self.groups[0].table, status=self.status)
        self.attend(seqs, row_ctx)

    def attend(self, seqs, row_ctx):
        B.indexer_topk(self.plan, self.qi, self.w, self.idx, self.groups[1].table, row_ctx, self.out["idx"], self.out["len"], self.ws, status=self.status, row_seq=seqs)
        more = dict(out_codes=self.out["codes"], out_scales=self.out["scales"], cos_sin=self.cs) if self.v4 else {}
        B.sparse_mla_prefill(self.plan, self.q, self.swa, self.groups[0].table, row_ctx, seqs, self.out["out"], self.ws, comp_cache=self.comp, comp_block_table=self.groups[1].table,
                             topk_idx=self.out["idx"], topk_len=self.out["len"], lse=self.out["lse"], status=self.status, **more)

    def whole(self, one_token=True):
        self.tables_step()
        self.path(ROWS, self.meta["seqs"], self.meta["positions"], self.meta["row_ctx"], one_token)

    def kept(self):
        return [t.clone() for t in (self.swa, self.comp, self.idx, *self.states)]


def compare(a, b, n):
    """a ran on padding; b on n rows, its attention's other rows standing for
    the first."""
    for x, y in zip(a.kept(), b.kept()):
        assert torch.equal(x, y)
    for k, t in a.out.items():
        if k in ("codes", "scales") and not a.v4:
            continue
        assert torch.equal(t[:n].view(torch.uint8), b.out[k][:n].view(torch.uint8)), k
        if k == "len":
            assert t[n:].eq(0).all()
        elif k == "idx":
            assert t[n:].eq(-1).all()
        else:
            assert t[n:].float().eq(77.0).all(), k
    assert B.read_device_status(a.status)[1] == 0 and B.read_device_status(b.status)[1] == 0


LENGTHS = [300, 1203, 7, 0, 129, 2000]


@pytest.mark.parametrize("v4,fp4,plan_ctx", [(True, False, CTX), (True, True, CTX), (False, False, CTX), (False, True, CTX),
                                             (True, False, 1 << 15), (False, True, 1 << 15), (True, False, 1 << 20)])
def test_a_captured_decode_step_with_idle_and_finished_sequences(v4, fp4, plan_ctx):
    """Contexts that the plan allows for choose among the indexer's launches."""
    pad, cut = (Step(v4, fp4, LENGTHS, plan_ctx=plan_ctx) for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pad.whole()
    lengths = list(LENGTHS)
    steps = [[1, 1, 1, 1, 1, 1], [1, 0, 1, 0, -1, 1], [0, 1, 0, 0, 0, 0], [0, 0, 0, 0, 0, 0], [1, -1, 1, 1, 0, 1], [0, 0, 1, 0, 0, -1]]
    for new in steps:
        for x in (pad, cut):
            x.computed.copy_(torch.tensor(lengths))
            x.new.copy_(torch.tensor(new))
            x.clear()
        graph.replay()
        n = sum(v > 0 for v in new)
        cut.tables_step()
        if n:
            m = cut.meta
            row = torch.tensor([min(t, n - 1) if t < n else 0 for t in range(ROWS)], device="cuda")
            cut.path(n, m["seqs"][row].contiguous(), m["positions"][row].contiguous(), m["row_ctx"][row].contiguous())
        torch.cuda.synchronize()
        assert pad.meta["seqs"][n:].eq(-1).all() and pad.meta["seqs"][:n].ge(0).all()
        compare(pad, cut, n)
        lengths = [0 if v < 0 else c + v for c, v in zip(lengths, new)]
        for x in (pad, cut):
            for g in x.groups:
                g.pool_in.copy_(g.pool_out)


@pytest.mark.parametrize("v4", [True, False])
def test_chunks_with_rows_behind_them(v4):
    """Several tokens a sequence, two launches of the compressor."""
    pad, cut = Step(v4, False, LENGTHS), Step(v4, False, LENGTHS)
    new = [5, 0, 3, 1, -1, 0]
    for x in (pad, cut):
        x.new.copy_(torch.tensor(new))
        x.clear()
    pad.whole(one_token=False)
    cut.tables_step()
    m, n = cut.meta, 9
    row = torch.tensor([t if t < n else 0 for t in range(ROWS)], device="cuda")
    cut.path(n, m["seqs"][row].contiguous(), m["positions"][row].contiguous(), m["row_ctx"][row].contiguous(), one_token=False)
    torch.cuda.synchronize()
    compare(pad, cut, n)


def test_rows_without_a_sequence_that_are_not_padding_are_flagged():
    x = Step(True, False, LENGTHS)
    for seq, at, ctx in ((-1, 5, 6), (-2, -1, 0), (S, 5, 6), (0, -1, None)):
        seqs, pos = i32(ROWS, fill=-1), i32(ROWS, fill=-1)
        seqs[3], pos[3] = seq, at
        x.status.zero_()
        B.cache_insert_rows(B.CACHE_V4, x.rows, seqs, pos, x.swa, x.groups[0].table, status=x.status)
        assert B.read_device_status(x.status)[1] == B.DEV_BAD_INDEX
        x.status.zero_()
        a = x.inputs[0]
        B.compress_insert(x.main_kind, 4, a["kv_score"], pos, seqs, a["ape"], a["rms_weight"], 1e-6, x.cs, x.states[0], x.comp, x.groups[1].table, S, status=x.status)
        assert B.read_device_status(x.status)[1] == B.DEV_BAD_INDEX
        if ctx is None:
            continue
        row_ctx = i32(ROWS)
        row_ctx[3] = ctx
        x.status.zero_()
        x.attend(seqs, row_ctx)
        assert B.read_device_status(x.status)[1] & B.DEV_BAD_INDEX
    x.status.zero_()
    B.inv_rope_fp8_quant(x.out["out"], i32(ROWS, fill=-1), x.cs, x.out["codes"], x.out["scales"], status=x.status)
    assert B.read_device_status(x.status)[1] == B.DEV_BAD_POSITION


def test_combined_indices_of_padding():
    topk, ln = i32(4, 8, fill=3), i32(4, fill=2)
    pos, seq = i32(4, fill=-1), i32(4, fill=-1)
    pos[0], seq[0] = 70, 0
    out, out_len, status = i32(4, 160, fill=-9), i32(4, fill=-9), i32(1)
    call = lambda: B.combine_topk_swa_indices(topk, ln, pos, seq, i32(1, fill=100), i32(1, fill=100), 128, 64, out, out_len, status=status)  # noqa: E731
    call()
    assert out_len.tolist() == [2 + 71, 0, 0, 0] and out[1:].eq(-9).all() and B.read_device_status(status)[1] == 0
    pos[2] = 4
    call()
    assert out_len.tolist() == [2 + 71, 0, -1, 0] and B.read_device_status(status)[1] == B.DEV_BAD_INDEX

"""The compiled torch binding of the attention path's calls: what it refuses, and its streams."""
import pytest

import block_quantized_token_format_gb300 as qg

torch = pytest.importorskip("torch")


def test_refusals_without_a_gpu():
    x = torch.zeros(4, 2, 128)
    with pytest.raises(TypeError, match="tensor"):
        qg.qg_qk_norm_rope([1.0], x, x, x)
    with pytest.raises(TypeError, match="tensor"):
        qg.qg_qk_norm_rope(None, x, x, x)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        qg.qg_qk_norm_rope(x.half(), x, x, x)
    with pytest.raises(ValueError, match="q: a CUDA"):
        qg.qg_qk_norm_rope(x, x, x, x)


@pytest.mark.gpu
class TestOnGpu:
    D, HQ, HK, N = 128, 4, 2, 3

    def setup_method(self):
        g = torch.Generator(device="cuda").manual_seed(5)
        draw = lambda h: torch.randn(self.N, h, self.D, device="cuda", generator=g)  # noqa: E731
        ints = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
        self.q, self.k, self.v = draw(self.HQ), draw(self.HK), draw(self.HK)
        self.pages = 4
        self.data = torch.zeros(qg.qg_cache_bytes(self.pages, 16, self.HK, self.D), dtype=torch.uint8, device="cuda")
        self.cache = qg.qg_cache(self.data, self.pages, 16, self.HK, self.D)
        self.ws = torch.zeros(qg.qg_attention_workspace_bytes(self.HQ, self.HK, self.D), dtype=torch.uint8, device="cuda")
        self.slots = ints([0, 1, 2], torch.int64)
        self.table, self.seq, self.cu = ints([[0, 1]]), ints([self.N]), ints([0, self.N])
        self.out = torch.zeros_like(self.q)

    def append(self, **kw):
        a = dict(cache=self.cache, k=self.k, v=self.v, slots=self.slots, norm=False)
        a.update(kw)
        qg.qg_cache_append(**a)

    def attend(self, **kw):
        a = dict(cache=self.cache, q=self.q, table=self.table, seq_len=self.seq, cu_new=self.cu, out=self.out,
                 workspace=self.ws, scale=0.1)
        a.update(kw)
        qg.qg_attention(**a)

    @pytest.mark.parametrize("name, make", [
        ("k", lambda s: s.k.bfloat16()), ("v", lambda s: s.v.bfloat16()), ("v", lambda s: s.v[:2]), ("v", lambda s: None),
        ("k", lambda s: s.k[..., ::2]), ("k", lambda s: s.k.transpose(0, 1)), ("slots", lambda s: s.slots.int()),
        ("slots", lambda s: s.slots[:2]), ("slots", lambda s: s.slots.cpu()), ("k_back", lambda s: s.k.bfloat16()),
        ("v_back", lambda s: s.v[:2]), ("k_weight", lambda s: torch.ones(64, device="cuda")), ("q", lambda s: s.q),
        ("cos_sin", lambda s: torch.ones(64, device="cuda")), ("positions", lambda s: s.seq)])
    def test_append_refuses(self, name, make):
        with pytest.raises(ValueError):
            self.append(**{name: make(self)})

    @pytest.mark.parametrize("name, make", [
        ("q", lambda s: s.q.bfloat16()), ("out", lambda s: None), ("out", lambda s: s.out[:2]), ("out", lambda s: s.out[:, :2]),
        ("table", lambda s: s.table[0]), ("table", lambda s: s.table.long()), ("table", lambda s: s.table.expand(2, 2)[:, :1]),
        ("table", lambda s: s.table[:0]), ("seq_len", lambda s: s.seq.long()), ("seq_len", lambda s: s.seq[:, None]),
        ("cu_new", lambda s: s.cu[:1]), ("span_mask", lambda s: s.seq), ("lse", lambda s: s.out[0, 0, :4]),
        ("lse", lambda s: s.out.bfloat16()), ("workspace", lambda s: s.ws.cpu()), ("max_new", lambda s: 1 << 40)])
    def test_attention_refuses(self, name, make):
        with pytest.raises(ValueError):
            self.attend(**{name: make(self)})

    def test_other_refusals(self):
        with pytest.raises(qg.QGError):
            self.attend(workspace=None)
        with pytest.raises(TypeError):
            self.attend(max_new="4")
        with pytest.raises(TypeError):
            self.attend(scale="1")
        with pytest.raises(TypeError):
            self.attend(cache=type("C", (), {"address": "x"})())
        with pytest.raises(ValueError):
            self.attend(cache=type("C", (), {"address": 0})())
        with pytest.raises(AttributeError):
            self.attend(stream="0")
        with pytest.raises(AttributeError):
            self.attend(cache=self.data)
        torch.cuda.synchronize()

    def test_streams_are_the_callers(self):
        """Default (torch's current), a Stream and its handle: the same work, ordered on that stream."""
        want = None
        side = torch.cuda.Stream()
        for stream in (None, side, side.cuda_stream):
            self.data.zero_()
            self.out.zero_()
            side.wait_stream(torch.cuda.current_stream())
            if stream is None:
                with torch.cuda.stream(side):
                    self.append()
                    self.attend()
            else:
                self.append(stream=stream)
                self.attend(stream=stream)
            side.synchronize()
            got = self.out.clone()
            assert got.abs().sum() > 0
            want = got if want is None else want
            assert torch.equal(got, want)

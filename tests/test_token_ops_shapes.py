"""What the binding makes of a tensor argument's shape, without a device: the
row stride of matrices whose rows are wider than the call's, and refusals of
tensors that the call would read or write at the wrong place."""
import pytest

import implicit_gemm_dgrad_gb300 as cdg

P = [1 << 24 << i for i in range(1, 14)]  # far-apart 16-byte aligned addresses


class FakeCuda:
    """Stands in for a contiguous CUDA tensor of a given shape."""
    is_cuda = True

    def __init__(self, *shape, esize=2, floating=True, at=1 << 24):
        self.shape, self.esize, self.floating, self.at = shape, esize, floating, at

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def element_size(self):
        return self.esize

    def is_contiguous(self):
        return True

    def is_floating_point(self):
        return self.floating

    def data_ptr(self):
        return self.at


class Recorder:
    """Stands in for the library: keeps the arguments of every call."""

    def __init__(self, real):
        self.real, self.calls = real, {}

    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return getattr(self.real, name)

        def call(*args):
            self.calls[name] = args
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    r = Recorder(cdg.load_library())
    monkeypatch.setattr(cdg, "load_library", lambda path=None: r)
    return r


def logprobs_ld(lib, logits, rows=4, vocab=100, **kw):
    cdg.token_logprobs(logits, P[1], P[2], None, rows, vocab, stream=0, **kw)
    return lib.calls["cdg_token_logprobs"][1]


def test_a_wider_contiguous_matrix_keeps_its_row_stride(lib):
    assert logprobs_ld(lib, FakeCuda(4, 128)) == 128
    assert logprobs_ld(lib, FakeCuda(4, 128), ld=128) == 128
    assert logprobs_ld(lib, FakeCuda(2, 2, 128)) == 128       # batch x positions x padded vocabulary
    assert logprobs_ld(lib, FakeCuda(6, 128)) == 128          # and more rows than the call takes
    assert logprobs_ld(lib, FakeCuda(1, 128), rows=1) == 128
    assert logprobs_ld(lib, FakeCuda(1, 128), rows=1, ld=100) >= 100  # one row: no stride to check
    cdg.token_logprobs_grad(FakeCuda(4, 128), P[1], P[2], None, P[3], None, FakeCuda(4, 104, at=P[4]), 4, 100, stream=0)
    args = lib.calls["cdg_token_logprobs_grad"]
    assert (args[1], args[13]) == (128, 104)
    cdg.embed(FakeCuda(10, 24), P[1], FakeCuda(4, 32, at=P[2]), 4, 10, 16, stream=0)
    args = lib.calls["cdg_embed"]
    assert (args[1], args[10]) == (24, 32)
    cdg.embed_grad(FakeCuda(4, 24), P[1], FakeCuda(10, 20, at=P[2]), P[3], 4, 10, 16, stream=0)
    args = lib.calls["cdg_embed_grad"]
    assert (args[1], args[10]) == (24, 20)


def test_dense_matrices_stay_dense(lib):
    assert logprobs_ld(lib, FakeCuda(4, 100)) == 100
    assert logprobs_ld(lib, FakeCuda(9, 100)) == 100          # a buffer for more rows
    assert logprobs_ld(lib, FakeCuda(2, 2, 100)) == 100
    assert logprobs_ld(lib, FakeCuda(400)) == 100
    assert logprobs_ld(lib, FakeCuda(1000)) == 100
    assert logprobs_ld(lib, FakeCuda(4, 10, 10)) == 100       # a row in two dimensions
    assert logprobs_ld(lib, FakeCuda(2, 200)) == 100          # as many elements as the call takes, in another shape


@pytest.mark.parametrize("shape,ld", [((3, 128), None), ((4, 128), 100), ((4, 128), 130), ((3, 3, 50), None),
                                      ((8, 60), None), ((5, 10, 11), None)])
def test_matrices_that_cannot_be_rows_of_the_call_are_refused(lib, shape, ld):
    with pytest.raises(ValueError, match="logits"):
        logprobs_ld(lib, FakeCuda(*shape), ld=ld)


def top_call(ids, logp, rows=4, top=20):
    cdg.token_logprobs(FakeCuda(rows, 100), None, None, P[1], rows, 100, top=top, top_ids=ids, top_logp=logp, stream=0)


@pytest.mark.parametrize("shape", [(4, 20), (6, 20), (2, 2, 20), (80,), (100,)])
def test_alternatives_are_written_dense(lib, shape):
    top_call(FakeCuda(*shape, esize=4, floating=False), FakeCuda(*shape, esize=4))
    assert "cdg_token_logprobs" in lib.calls


@pytest.mark.parametrize("shape", [(4, 32), (2, 2, 32), (4, 21)])
def test_alternatives_of_another_width_are_refused(lib, shape):
    """The alternatives' rows are dense: into a wider tensor they would be written side by side, not at its rows."""
    good = (4, 20)
    with pytest.raises(ValueError, match="top_ids"):
        top_call(FakeCuda(*shape, esize=4, floating=False), FakeCuda(*good, esize=4))
    with pytest.raises(ValueError, match="top_logp"):
        top_call(FakeCuda(*good, esize=4, floating=False), FakeCuda(*shape, esize=4))
    top_call(FakeCuda(1, 32, esize=4, floating=False), FakeCuda(1, 32, esize=4), rows=1)  # a single row has no stride


def test_alternatives_without_top_are_the_librarys_refusal():
    with pytest.raises(cdg.CdgError) as e:
        top_call(FakeCuda(4, 20, esize=4, floating=False), FakeCuda(4, 20, esize=4), top=0)
    assert e.value.status == 1


def typed(name, *shape, at=1 << 24):
    """A contiguous stand-in that says its type, as torch's tensors do."""
    torch = pytest.importorskip("torch")
    dt = getattr(torch, name)
    t = FakeCuda(*shape, esize=dt.itemsize, floating=dt.is_floating_point, at=at)
    t.dtype = dt
    return t


@pytest.mark.parametrize("dtype,wrong", [("bf16", "float16"), ("f16", "bfloat16"), ("bf16", "int16"), ("f32", "int32")])
def test_matrices_of_another_type_are_refused(lib, dtype, wrong):
    """Elements of the right size and the wrong type would be read as other numbers."""
    right = {"f16": "float16", "bf16": "bfloat16", "f32": "float32"}[dtype]
    with pytest.raises(ValueError, match="logits.*type"):
        cdg.token_logprobs(typed(wrong, 4, 100), P[1], P[2], None, 4, 100, dtype, stream=0)
    with pytest.raises(ValueError, match="dlogits.*type"):
        cdg.token_logprobs_grad(typed(right, 4, 100), P[1], P[2], None, P[3], None, typed(wrong, 4, 100), 4, 100, dtype, stream=0)
    with pytest.raises(ValueError, match="table.*type"):
        cdg.embed(typed(wrong, 10, 16), P[1], P[2], 4, 10, 16, dtype, stream=0)
    with pytest.raises(ValueError, match="out.*type"):
        cdg.embed(P[0], P[1], typed(wrong, 4, 16), 4, 10, 16, dtype, stream=0)
    with pytest.raises(ValueError, match="dout.*type"):
        cdg.embed_grad(typed(wrong, 4, 16), P[1], P[2], P[3], 4, 10, 16, dtype, stream=0)
    with pytest.raises(ValueError, match="dtable.*type"):
        cdg.embed_grad(P[0], P[1], typed(wrong, 10, 16), P[3], 4, 10, 16, dtype, stream=0)
    p = cdg.muon_plan_host(8, 16, dtype=dtype)
    ws = typed("uint8", p.workspace_bytes)
    for a, b in ((typed(wrong, 8, 16), P[1]), (P[0], typed(wrong, 8, 16))):
        with pytest.raises(ValueError, match="[UO] .*type"):
            p.orthogonalize(a, b, ws)
    with pytest.raises(ValueError, match="G.*type"):
        p.step(P[0], typed(wrong, 8, 16), P[1], P[2], P[3], ws, lr=0.1)


def test_fp32_arguments_and_token_numbers_have_their_types(lib):
    logits = typed("bfloat16", 4, 100)
    for bad in ("int32",):
        with pytest.raises(ValueError, match="logp.*type"):
            cdg.token_logprobs(logits, P[1], typed(bad, 4), None, 4, 100, stream=0)
        with pytest.raises(ValueError, match="entropy.*type"):
            cdg.token_logprobs(logits, None, None, P[2], 4, 100, entropy=typed(bad, 4), stream=0)
        with pytest.raises(ValueError, match="g_logp.*type"):
            cdg.token_logprobs_grad(logits, P[1], P[2], None, typed(bad, 4), None, P[4], 4, 100, stream=0)
    with pytest.raises(ValueError, match="top_ids.*type"):
        top_call(typed("float32", 4, 20), typed("float32", 4, 20))
    with pytest.raises(ValueError, match="token numbers"):
        cdg.embed(P[0], typed("complex64", 4), P[2], 4, 10, 16, stream=0)
    with pytest.raises(ValueError, match="dtable.*type"):
        cdg.embed_grad(P[0], P[1], typed("int32", 10, 16), P[3], 4, 10, 16, out_f32=True, stream=0)
    p = cdg.muon_plan_host(8, 16)
    with pytest.raises(ValueError, match="M_out.*type"):
        p.step(P[0], P[1], P[2], P[3], typed("int32", 8, 16), typed("uint8", p.workspace_bytes), lr=0.1)


def test_the_right_types_pass(lib):
    for dtype, name in (("f16", "float16"), ("bf16", "bfloat16"), ("f32", "float32"), (cdg.BF16, "bfloat16")):
        for index in ("int32", "int64"):
            cdg.token_logprobs(typed(name, 4, 100), typed(index, 4), typed("float32", 4), None, 4, 100, dtype, top=2,
                               top_ids=typed("int32", 4, 2), top_logp=typed("float32", 4, 2), stream=0)
            cdg.embed_grad(typed(name, 4, 16), typed(index, 4), typed("float32", 10, 16), P[3], 4, 10, 16, dtype, out_f32=True,
                           stream=0)

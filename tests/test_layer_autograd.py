"""What autograd is told about the layer operators, which record nothing for
it: tensors that a call writes count as modified in place, and a call that
cuts a gradient off says so."""

import warnings

import pytest

kb = pytest.importorskip("blockwise_bit_codebook_amd")
torch = pytest.importorskip("torch")


def test_a_gradient_that_is_cut_off_is_said():
    # the arguments are on the host, so every call ends with its refusal
    h = torch.zeros(4, 2, 32, requires_grad=True)
    x = torch.zeros(4, 32, requires_grad=True)
    w = torch.zeros(32, requires_grad=True)
    t, pos, i8 = torch.zeros(8, 32), torch.zeros(4, dtype=torch.int64), torch.zeros(4, 32, dtype=torch.int8)
    d = h.detach()
    calls = [lambda: kb.quantize_rows_int8(x), lambda: kb.linear_int8(i8, w, i8, w), lambda: kb.rope(h, pos, t),
             lambda: kb.linear_int8_dynamic(x, i8, w.detach()), lambda: kb.rope(d, pos, t, out=h),
             lambda: kb.qk_norm_rope(d, d, w, w, pos, t), lambda: kb.append_kv_paged(d, d, pos, h[None], d[None]),
             lambda: kb.qk_norm_rope_backward(d, h, d, d, t[0], t[0], pos, t)]
    for i, call in enumerate(calls):
        with pytest.warns(UserWarning, match="requires a gradient") as seen, pytest.raises(ValueError, match="GPU"):
            call()
        assert seen[0].filename == __file__, i
        with warnings.catch_warnings():  # nothing to say where nothing is recorded
            warnings.simplefilter("error")
            with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
                call()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError, match="GPU"):
            kb.rope(d, pos, t)
        with pytest.raises(UserWarning):  # as an error it comes before the call's own checks
            kb.rope(h, pos, t)


@pytest.mark.gpu
def test_written_tensors_count_as_modified():
    dev = torch.device("cuda:0")
    x = torch.randn(6, 64, device=dev)
    codes = torch.empty(6, 64, dtype=torch.int8, device=dev)
    scale, out = torch.empty(6, device=dev), torch.empty(6, 6, device=dev)
    h = torch.randn(6, 2, 64, device=dev)
    q, k, gq, gk = (h.clone() for _ in range(4))
    pos = torch.arange(6, device=dev)
    w = torch.ones(64, device=dev)
    table = torch.empty(8, 64, device=dev)
    kc, vc = (torch.zeros(2, 4, 2, 64, device=dev) for _ in range(2))
    freq, _ = kb.rope_frequencies(64)
    calls = [(lambda: kb.rope_table(freq, 8, out=table), [table]),
             (lambda: kb.quantize_rows_int8(x, codes=codes, scale=scale), [codes, scale]),
             (lambda: kb.linear_int8(codes, scale, codes, scale, dtype=torch.float32, out=out), [out]),
             (lambda: kb.linear_int8_dynamic(x, codes, scale, out=out), [out]),
             (lambda: kb.rope(h, pos, table, out=h), [h]),
             (lambda: kb.qk_norm_rope(q, k, w, w, pos, table, q_out=q, k_out=k), [q, k]),
             (lambda: kb.qk_norm_rope_backward(gq, gk, q, k, w, w, pos, table, dq=gq, dk=gk), [gq, gk]),
             (lambda: kb.append_kv_paged(q, k, pos, kc, vc), [kc, vc])]
    everything = [x, codes, scale, out, h, q, k, gq, gk, pos, w, table, kc, vc]
    for i, (call, written) in enumerate(calls):
        before = [t._version for t in everything]
        call()
        for t, v in zip(everything, before):
            assert (t._version > v) == any(t is o for o in written), i
    before = h._version  # a refused call writes nothing
    with pytest.raises(kb.KbitError):
        kb.qk_norm_rope(h, k, w, w, pos, table, eps=-1.0, q_out=h, k_out=k)
    assert h._version == before
    with torch.inference_mode():
        inside = torch.randn(6, 2, 64, device=dev)
        kb.rope(inside, pos, table, out=inside)
    kb.rope(inside, pos, table, out=inside)  # an inference tensor has no version


@pytest.mark.gpu
def test_a_backward_pass_over_rotated_values_is_refused():
    dev = torch.device("cuda:0")
    freq, _ = kb.rope_frequencies(64)
    table, pos = kb.rope_table(freq, 8), torch.arange(6, device=dev)
    x = torch.randn(6, 2, 64, device=dev, requires_grad=True)
    y = x * 2.0
    loss = (y * y).sum()  # saves y
    with torch.no_grad():
        kb.rope(y, pos, table, out=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()

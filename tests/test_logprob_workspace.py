"""The workspace of logprob_rows serves every smaller call: fewer rows (which
are cut into more parts), shorter rows, fewer alternatives."""
import numpy as np
import pytest

import moe_expert_ffn_q8_amd as q

lib = q.raw
VOCABS = (1, 1000, 16384, 32767, 32768, 50257, 131071, 262144, 700001, 1048576, 1 << 30)


def _parts(m, v):
    """Parts of a row, as the calls cut them: 1024 workgroups, of 16384 logits at
    least, none of a part from 512 rows on."""
    return 1 if m >= 512 else max(1, min(1024 // m, v // 16384, 64))


@pytest.mark.parametrize("v", VOCABS)
def test_serves_fewer_rows(v):
    for n_top in (0, 1, 20, 64):
        if n_top > v:
            continue
        need, before = 256, 0
        for m in list(range(1, 600)) + [1021, 4096, 1 << 24]:
            parts = _parts(m, v)
            need = max(need, m * parts * (8 * n_top + 12) if parts > 1 else 0)
            have = lib.logprob_workspace_bytes(m, v, n_top)
            assert have >= need and have >= before, (m, v, n_top)
            before = have
        assert before <= 1024 * (8 * n_top + 12) + 255


def test_serves_smaller_calls():
    for m in (1, 7, 300, 2000):
        for n_top in (0, 1, 20, 64):
            sizes = [lib.logprob_workspace_bytes(m, v, n_top) for v in VOCABS if v >= n_top]
            assert sizes == sorted(sizes)
        sizes = [lib.logprob_workspace_bytes(m, 262144, n_top) for n_top in range(65)]
        assert sizes == sorted(sizes)


@pytest.mark.gpu
def test_one_workspace_for_all_batches():
    """A server's workspace, made for its largest batch."""
    import torch

    import i8_ref
    import synth
    from gpu_cases import to_gpu
    v, n_top = 70001, 20
    rng = synth.rng("lpserver")
    x = (rng.normal(size=(520, v)) * 2.5).astype(np.float32)
    ws = q.logprob_workspace(600, v, n_top, "cuda")
    guard = torch.full((ws.numel() + 4096,), 77, dtype=torch.uint8, device="cuda")
    ws = guard[:ws.numel()]
    logits = to_gpu(x)
    for m in (520, 1, 3, 8, 64, 255, 256, 300, 511):
        out = q.logprob_rows(logits[:m], n_top=n_top, ws=ws)
        few = slice(max(0, m - 4), m)
        ref = i8_ref.logprobs(x[few].astype(np.float64), None, n_top)
        i8_ref.assert_logprobs(out._replace(lse=out.lse[few], entropy=out.entropy[few],
                                            top_ids=out.top_ids[few],
                                            top_logprobs=out.top_logprobs[few]), ref)
    assert bool((guard[ws.numel():] == 77).all())

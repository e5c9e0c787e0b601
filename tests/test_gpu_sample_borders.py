"""Draws and cuts whose target lies between two roundings of one cumulative mass.

A row's masses are added up by a scan, whose threads form the same sum along different
paths.  In these rows (the bits of their fp32 logits) the last bin before the middle of
the mass and a bin without tokens right behind it, in the next thread's share, come out
half an ulp apart, and the target lies in between: u or top_p of one half is the mass of
the first tokens to the last bit.  Found by following the scan's additions on the CPU, for
the 512 threads of a work-group per row and the 1024 of the rows that are cut into pieces.

At such a border either neighbour is a right answer in 53 bits; none is not.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BELOW_1 = 1 - 2.0 ** -24

# target u M: a mass has to exceed it
DRAW = {
    512: [
        [0x00000000, 0xbf39ac59, 0xbfb79bd0, 0xbfcd9142, 0xbfcccd79, 0xbfcd05db, 0xbfce8def,
     0xbfcc9c44, 0xbfcf7770, 0xbfcbf625, 0xbfcb416f, 0xc00c4edb, 0xc18d11f6, 0xc200b097],
        [0x00000000, 0xbf32fb47, 0xbf421fb7, 0xbfb97748, 0xbfcc3024, 0xbfcf6cdc, 0xbfcccd9e,
     0xbfcabe62, 0xbfcc361f, 0xbfcb7068, 0xbfca8f5d, 0xbfcc643d, 0xbfcd2366, 0xbfce1cd1, 0xbfde04c0,
     0xc18e3744, 0xc1f85f1d],
        [0x00000000, 0xbf375511, 0xbfb323ab, 0xbfcd0a71, 0xbfcd8292, 0xbfcbb185, 0xbfca7d1b,
     0xbfcf10d9, 0xbfcfa236, 0xbfcdcaae, 0xbfce5223, 0xc0037e55, 0xc18e5bc7, 0xc1fa99eb],
        [0x00000000, 0xbf3f43ac, 0xbf330d47, 0xbfbc1859, 0xbfcc7461, 0xbfca6440, 0xbfcd740f,
     0xbfca5832, 0xbfcd3dda, 0xbfcd0dae, 0xbfcfa02d, 0xbfcd88d6, 0xbfca24fd, 0xbfcb00cc, 0xbfdfd85f,
     0xc18e8127, 0xc1fd4b03],
    ],
    1024: [
        [0x00000000, 0xbf37786b, 0xbf38b825, 0xbfb49148, 0xbfc299ea, 0xbfc0f049, 0xbfc20851,
     0xbfbf01d6, 0xbfbefcbf, 0xbfbfe67b, 0xbfc2dc2b, 0xbfc1486e, 0xbfc09342, 0xbfc244b6, 0xc0a9228d,
     0xc19f9b38, 0xc20aa123],
        [0x00000000, 0xbf35ce7b, 0xbf35c41c, 0xbfb4d678, 0xbfb1e752, 0xbfbf091e, 0xbfbfeaf5,
     0xbfbfa0c3, 0xbfc0bca2, 0xbfbef186, 0xbfbe9def, 0xbfbf8f22, 0xbfbf3f9a, 0xbfc0e240, 0xbfbec649,
     0xbfc411e1, 0xc079ec8d, 0xc1aa3d09],
        [0x00000000, 0xbf333f32, 0xbf344f8d, 0xbfb4ac6f, 0xbfb40431, 0xbfbf55c8, 0xbfc1a903,
     0xbfc4b728, 0xbfc19cc2, 0xbfc08f98, 0xbfbf83b8, 0xbfc34acd, 0xbfc33be9, 0xbfc199ed, 0xbfc2eec9,
     0xbfc1d627, 0xc033cbff, 0xc195e8bb, 0xc202d886],
        [0x00000000, 0xbf377c49, 0xbf3984f6, 0xbfb3db9d, 0xbfc26fc6, 0xbfc1c4ef, 0xbfc1cf7d,
     0xbfc2efdc, 0xbfc16ff6, 0xbfc1f139, 0xbfc198fe, 0xbfc47d26, 0xbfc2fa38, 0xbfc41566, 0xc05ed115,
     0xc1abd764],
    ],
}
# target top_p M1: a mass has to reach it
REACH = {
    512: [
        [0x00000000, 0xbf39ac59, 0xbfb79bd0, 0xbfcd9142, 0xbfcccd79, 0xbfcd05db, 0xbfce8def,
     0xbfcc9c44, 0xbfcf7770, 0xbfcbf625, 0xbfcb416f, 0xc00c4edb, 0xc18d11f6, 0xc20086ca],
        [0x00000000, 0xbf32fb47, 0xbf421fb7, 0xbfb97748, 0xbfcc3024, 0xbfcf6cdc, 0xbfcccd9e,
     0xbfcabe62, 0xbfcc361f, 0xbfcb7068, 0xbfca8f5d, 0xbfcc643d, 0xbfcd2366, 0xbfce1cd1, 0xbfde04c0,
     0xc18e3744, 0xc1f8287f],
        [0x00000000, 0xbf375511, 0xbfb323ab, 0xbfcd0a71, 0xbfcd8292, 0xbfcbb185, 0xbfca7d1b,
     0xbfcf10d9, 0xbfcfa236, 0xbfcdcaae, 0xbfce5223, 0xc0037e55, 0xc18e5bc7, 0xc1fa75ab],
        [0x00000000, 0xbf3f43ac, 0xbf330d47, 0xbfbc1859, 0xbfcc7461, 0xbfca6440, 0xbfcd740f,
     0xbfca5832, 0xbfcd3dda, 0xbfcd0dae, 0xbfcfa02d, 0xbfcd88d6, 0xbfca24fd, 0xbfcb00cc, 0xbfdfd85f,
     0xc18e8127, 0xc1fce717],
    ],
    1024: [
        [0x00000000, 0xbf37786b, 0xbf38b825, 0xbfb49148, 0xbfc299ea, 0xbfc0f049, 0xbfc20851,
     0xbfbf01d6, 0xbfbefcbf, 0xbfbfe67b, 0xbfc2dc2b, 0xbfc1486e, 0xbfc09342, 0xbfc244b6, 0xc0a9228d,
     0xc19f9b38, 0xc207db5a],
        [0x00000000, 0xbf35ce7b, 0xbf35c41c, 0xbfb4d678, 0xbfb1e752, 0xbfbf091e, 0xbfbfeaf5,
     0xbfbfa0c3, 0xbfc0bca2, 0xbfbef186, 0xbfbe9def, 0xbfbf8f22, 0xbfbf3f9a, 0xbfc0e240, 0xbfbec649,
     0xbfc411e1, 0xc079ec8d, 0xc1aa3d08],
        [0x00000000, 0xbf333f32, 0xbf344f8d, 0xbfb4ac6f, 0xbfb40431, 0xbfbf55c8, 0xbfc1a903,
     0xbfc4b728, 0xbfc19cc2, 0xbfc08f98, 0xbfbf83b8, 0xbfc34acd, 0xbfc33be9, 0xbfc199ed, 0xbfc2eec9,
     0xbfc1d627, 0xc033cbff, 0xc195e8bb, 0xc2024fca],
        [0x00000000, 0xbf377c49, 0xbf3984f6, 0xbfb3db9d, 0xbfc26fc6, 0xbfc1c4ef, 0xbfc1cf7d,
     0xbfc2efdc, 0xbfc16ff6, 0xbfc1f139, 0xbfc198fe, 0xbfc47d26, 0xbfc2fa38, 0xbfc41566, 0xc05ed115,
     0xc1abd763],
    ],
}


@pytest.fixture(scope="module")
def lg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rank_gradient_sketching_amd as m
    return m


def place(bits, threads):
    """(logits [1, V] on the GPU, positions of the tokens in descending order, their
    probabilities): spread over a row of otherwise masked tokens, long enough to be cut into
    pieces or not."""
    z = np.array(bits, np.uint32).view(np.float32)
    V = 16384 if threads == 1024 else 160
    at = (np.arange(len(z)) * 37 + 5) % V
    row = torch.full((1, V), -float("inf"))
    row[0, torch.from_numpy(at)] = torch.from_numpy(z)
    order = np.argsort(-z, kind="stable")
    p = np.exp(z[order].astype(np.float64))
    return row.cuda(), at[order], p / p.sum()


@pytest.mark.parametrize("threads", DRAW)
@pytest.mark.parametrize("i", range(4))
@pytest.mark.parametrize("more", [1, 3])
def test_draw_between_two_roundings(lg, threads, i, more):
    z, at, p = place(DRAW[threads][i], threads)
    assert (lg.sample_tokens_ws_bytes(more, z.shape[1]) > 0) == (threads == 1024)
    c = int(np.argmin(np.abs(np.cumsum(p) - 0.5)))      # the border lies behind this token
    assert abs(np.cumsum(p)[c] - 0.5) < 1e-12
    got = lg.sample_tokens(z.repeat(more, 1), torch.full((more,), 0.5, device="cuda"))
    for t in range(more):
        token, kept = got.token[t].item(), got.kept[t].item()
        assert token in (at[c], at[c + 1]) and kept == len(p), (token, kept)
        want = np.log(p[c if token == at[c] else c + 1])
        assert abs(got.logp[t].item() - want) <= U * abs(want) + 1e-7
        assert got.logq[t].item() == got.logp[t].item()


@pytest.mark.parametrize("threads", REACH)
@pytest.mark.parametrize("i", range(4))
def test_cut_between_two_roundings(lg, threads, i):
    z, at, p = place(REACH[threads][i], threads)
    c = int(np.argmin(np.abs(np.cumsum(p) - 0.5)))
    assert abs(np.cumsum(p)[c] - 0.5) < 1e-12
    u = torch.tensor([0.0, BELOW_1], device="cuda")
    got = lg.sample_tokens(z.repeat(2, 1), u, top_p=0.5)
    kept = got.kept[0].item()
    assert kept in (c + 1, c + 2) and got.kept[1].item() == kept
    assert got.token.tolist() == [at[0], at[kept - 1]]
    for t, j in ((0, 0), (1, kept - 1)):
        want = np.log(p[j])
        assert abs(got.logp[t].item() - want) <= U * abs(want) + 1e-7
        want = np.log(p[j] / p[:kept].sum())
        assert abs(got.logq[t].item() - want) <= U * abs(want) + 1e-7

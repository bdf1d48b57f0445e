"""The largest batches that are accepted: tokens, sequences, heads of one."""
import numpy as np
import pytest
import torch

import block_quantized_amd as Q

pytestmark = pytest.mark.gpu


def check_rows(got, q, k, v, rows, keys_of, scale):
    """Rows of one head against the definition in 64 bits, within 2^-18 of the norm."""
    for r in rows:
        j = keys_of(r)
        w = torch.exp(scale * (k[j].double() @ q[r].double()))
        want = (w / w.sum()) @ v[j].double()
        assert (got[r].double() - want).norm() <= 2.0 ** -18 * want.norm(), r


@pytest.mark.parametrize("algo", [1, 2])
def test_tokens(algo):
    # 2^23 - 1 tokens at once, each with the 20 keys before it, stored by the same call
    N, D, page = 2 ** 23 - 1, 64, 4096
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("not enough free memory")
    g = torch.Generator(device="cuda").manual_seed(3)
    n_pages = -(-N // page)
    c = Q.KVCache.allocate(Q.QMM_F16, 1, D, page, n_pages)
    x = [torch.randn(N, 1, D, generator=g, device="cuda").half().float() for _ in range(3)]
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    b = Q.KVBatch(i([0, N]), i([N]), torch.randperm(n_pages, generator=g, device="cuda").int()[None], N, max_kv=N)
    Q.kv_append(c, b, x[1], x[2])
    got = Q.attn(c, b, x[0], window=20, algo=algo)
    q, k, v = (y[:, 0] for y in x)
    rows = [0, 1, 19, 20, 4095, 4096, 2 ** 22 - 1, 2 ** 22 + 77, N - 129, N - 2, N - 1]
    check_rows(got[:, 0], q, k, v, rows, lambda r: torch.arange(max(0, r - 19), r + 1, device="cuda"), float(np.float32(D ** -0.5)))
    del x, got, q, k, v
    torch.cuda.empty_cache()


@pytest.mark.parametrize("algo", [1, 2])
def test_sequences(algo):
    # 65536 sequences of one to three tokens, a page each
    S, D, page = 65536, 64, 16
    g = torch.Generator(device="cuda").manual_seed(4)
    new = torch.randint(0, 2, (S,), generator=g, device="cuda")
    length = new + torch.randint(0, 3, (S,), generator=g, device="cuda")
    q_start = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), new.cumsum(0)])
    N = int(q_start[-1])
    c = Q.KVCache.allocate(Q.QMM_F16, 1, D, page, S)
    c.k.normal_(generator=g), c.v.normal_(generator=g)
    table = torch.randperm(S, generator=g, device="cuda")
    b = Q.KVBatch(q_start.int(), length.int(), table.int()[:, None].contiguous(), N, max_kv=4)
    q = torch.randn(N, 1, D, generator=g, device="cuda")
    got = Q.attn(c, b, q, algo=algo)
    seqs = [s for s in list(range(0, 70)) + list(range(32700, 32800)) + list(range(S - 70, S)) if new[s]]
    for s in seqs:
        r, n, p = int(q_start[s]), int(length[s]), int(table[s])
        check_rows(got[:, 0], q[:, 0], c.k[p, 0], c.v[p, 0], [r], lambda _: torch.arange(n, device="cuda"), float(np.float32(D ** -0.5)))


@pytest.mark.parametrize("algo", [1, 2])
def test_heads(algo):
    # 4096 query heads of one key-value head: 256 and 32 row tiles of a token
    g = torch.Generator(device="cuda").manual_seed(5)
    c = Q.KVCache.allocate(Q.QMM_BF16, 1, 64, 16, 20)
    c.k.normal_(generator=g), c.v.normal_(generator=g)
    table = torch.randperm(20, generator=g, device="cuda").int()[None]
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.randn(2, 4096, 64, generator=g, device="cuda")
    got = Q.attn(c, Q.KVBatch(i([0, 2]), i([311]), table, 2), q, algo=algo)
    k, v = (x[table[0].long(), 0].reshape(-1, 64)[:311].double() for x in (c.k, c.v))
    for t, n in ((0, 310), (1, 311)):
        w = torch.softmax(q[t].double() @ k[:n].T * float(np.float32(0.125)), 1)
        want = w @ v[:n]
        assert ((got[t].double() - want).norm(dim=1) <= 2.0 ** -18 * want.norm(dim=1)).all()

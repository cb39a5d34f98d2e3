"""The chunk form of the sequence operators in fp32 on the CPU, every operand a
sum of bf16 parts (test infrastructure): what a kernel's results would be with
`parts` of them, for fp32 inputs and a scalar gate, one sequence of one head.
"""
import torch

C = 64


def split(x, n):
    out = []
    for _ in range(n):
        out.append(x.bfloat16().float())
        x = x - out[-1]
    return out


def product(a, b, parts):
    """a @ b from the products of parts (i, j), i + j <= 2, small ones first."""
    a, b = split(a, parts), split(b.contiguous(), parts)
    y = torch.zeros(a[0].shape[0], b[0].shape[1])
    for t in (2, 1, 0):
        for i in range(parts):
            if 0 <= t - i < parts:
                y = y + a[i] @ b[t - i]
    return y


def _decays(alpha):
    n = len(alpha)
    L = torch.zeros(n, n)
    for j in range(n):
        L[j, j] = 1.0
        for i in range(j + 1, n):
            L[i, j] = L[i - 1, j] * alpha[i]
    return L


def forward_backward(q, k, v, beta, alpha, S, do, dS, parts):
    """o, S, dq, dk, dv, dbeta, dalpha, dS0 of tensors [tokens, 128] and [tokens], states [128, 128]."""
    P_ = lambda a, b: product(a, b, parts)  # noqa: E731
    kept, out = [], []
    for c in range(0, len(q), C):
        Q, K, V, be, al = (x[c:c + C] for x in (q, k, v, beta, alpha))
        L = _decays(al)
        gam, kap = torch.cumprod(al, 0), L[-1] * be
        qk, kk = P_(Q, K.T), P_(K, K.T)
        M, P = torch.tril(L * be * kk, -1), torch.tril(L * be * qk)
        T = torch.linalg.solve_triangular(torch.eye(len(Q)) + M, torch.eye(len(Q)), upper=False)
        U = P_(T, V - gam[:, None] * P_(K, S))
        out.append(gam[:, None] * P_(Q, S) + P_(P, U))
        kept.append((c, Q, K, be, al, L, gam, kap, qk, kk, P, T, U, S))
        S = gam[-1] * S + P_(K.T, kap[:, None] * U)
    end, G = S, dS
    grads = []
    for c, Q, K, be, al, L, gam, kap, qk, kk, P, T, U, S0 in reversed(kept):
        n, dO = len(Q), do[c:c + C]
        dX = P_(T.T, P_(P.T, dO) + kap[:, None] * P_(K, G))
        D1, D2 = P_(dO, U.T), -P_(dX, U.T)
        E1, E2 = torch.tril(L * be * D1), torch.tril(L * be * D2, -1)
        Z1, Z2, Z3 = P_(dO, S0.T), P_(dX, S0.T), P_(U, G.T)
        dQ = gam[:, None] * Z1 + P_(E1, K)
        dK = -gam[:, None] * Z2 + kap[:, None] * Z3 + P_(E1.T, Q) + P_(E2 + E2.T, K)
        W = torch.tril(D1 * qk) + torch.tril(D2 * kk, -1)
        kz = (K * Z3).sum(1)
        dbeta = (L * W).sum(0) + L[-1] * kz
        # dL's columns: the state's, then the tokens'; the last row holds what comes from the chunk's end
        dL = torch.cat([((Q * Z1).sum(1) - (K * Z2).sum(1))[:, None], torch.tril(be * W, -1)], 1)
        dL[-1] = dL[-1] + torch.cat([(G * S0).sum().view(1), be * kz])
        before = torch.cat([gam[:, None], L], 1)  # decays from a column's place to token t
        dalpha, F = torch.zeros(n), torch.zeros(n + 1)
        for t in reversed(range(n)):
            F = dL[t] + (al[t + 1] if t + 1 < n else 0.0) * F
            to = torch.cat([torch.ones(1), torch.zeros(n)]) if t == 0 else before[t - 1]
            use = torch.arange(n + 1) <= t  # columns before token t
            dalpha[t] = (to * F)[use].sum()
        grads.append((dQ, dK, dX, dbeta, dalpha))
        G = gam[-1] * G + P_(Q.T, gam[:, None] * dO) - P_(K.T, gam[:, None] * dX)
    return (torch.cat(out), end, *[torch.cat(x) for x in zip(*reversed(grads))], G)

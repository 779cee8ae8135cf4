"""fp64 oracle of linear attention with a decay per head: S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t,
token by token, and its gradients by the recurrence of the state's adjoint.  Test infrastructure only.

q, k [T, H, dk], v [T, H, dv], g [T, H] (log-decays), states [H, dk, dv]; shared heads are repeated by the caller
(repeat_heads) and their gradients summed (sum_heads)."""
import numpy as np


def repeat_heads(x, H):
    return np.repeat(np.asarray(x, np.float64), H // x.shape[1], axis=1)


def sum_heads(x, Hx):
    T, H = x.shape[:2]
    return x.reshape(T, Hx, H // Hx, -1).sum(2)


def forward(q, k, v, g, S0, scale=1.0):
    """(o [T, H, dv], final state)."""
    T, H, _ = q.shape
    S = np.array(S0, np.float64)
    o = np.zeros((T, H, v.shape[2]))
    a = np.exp(g)
    for t in range(T):
        S = a[t][:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
        o[t] = scale * np.einsum("hkv,hk->hv", S, q[t])
    return o, S


def backward(q, k, v, g, S0, grad_o, grad_final, scale=1.0):
    """Gradients of sum(o * grad_o) + sum(S_T * grad_final): dict of q, k, v, g, initial_state."""
    T = q.shape[0]
    a = np.exp(g)
    states = [np.array(S0, np.float64)]
    for t in range(T):
        states.append(a[t][:, None, None] * states[-1] + k[t][:, :, None] * v[t][:, None, :])
    L = np.array(grad_final, np.float64)
    d = {"q": np.zeros_like(q), "k": np.zeros_like(k), "v": np.zeros_like(v), "g": np.zeros_like(g)}
    for t in range(T - 1, -1, -1):
        L = L + scale * q[t][:, :, None] * grad_o[t][:, None, :]  # adjoint of S_t
        d["q"][t] = scale * np.einsum("hkv,hv->hk", states[t + 1], grad_o[t])
        d["k"][t] = np.einsum("hkv,hv->hk", L, v[t])
        d["v"][t] = np.einsum("hkv,hk->hv", L, k[t])
        L = a[t][:, None, None] * L
        d["g"][t] = (L * states[t]).sum((1, 2))
    d["initial_state"] = L
    return d

"""A recurrent student distilled from a teacher's top logits over prioritised
replay, with every operator of include/per_train.h next to the sum tree:

  actor    per_scan_step runs the student one token at a time; the feature rows
           go to the ring in 8 bits (per_rows_write), the teacher's top logits
           beside them, and the slots enter the sum tree at the running max;
  learner  per_sample draws slots and IS weights, per_rows_read gives the
           sequences behind them, per_scan_forward / per_scan_backward and
           per_distill the loss and gradients; the row losses become the new
           priorities (per_update), and the recurrent state at each sampled
           slot is stored again with the present weights (per_rows_write_at).

    python3 examples/replay_distill.py [--steps 200]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sum_tree_sampling_amd as per  # noqa: E402

DIM, HIDDEN, VOCAB, K = 64, 128, 500, 16     # feature row, student's state, tokens, teacher entries
CAPACITY, ACTORS, BATCH, WINDOW = 1 << 14, 64, 64, 32
TEMPERATURE = 2.0


class Replay:
    """The ring: slot s holds an actor's feature row, episode flag, the
    student's state before it and the teacher's top logits after it."""

    def __init__(self):
        self.tree = per.PerBuffer(CAPACITY, max_batch=4096)
        self.rows = per.rows_alloc(CAPACITY, DIM, group=0)
        self.states = per.rows_alloc(CAPACITY, HIDDEN, dtype=torch.int8, group=64)
        self.claims = torch.zeros(CAPACITY, dtype=torch.int32, device="cuda")
        self.begins = torch.ones(CAPACITY, dtype=torch.bool, device="cuda")
        self.tidx = torch.full((CAPACITY, K), -1, dtype=torch.int32, device="cuda")  # no entry: no loss
        self.tlogit = torch.zeros(CAPACITY, K, device="cuda")
        self.tlse = torch.zeros(CAPACITY, device="cuda")

    def add(self, rows, states, begins, top):
        """One actor's episode: consecutive slots, so that sequences lie in the ring."""
        n, at = rows.shape[0], self.tree.cursor
        per.per_rows_write(*self.rows, rows, at, group=0)
        per.per_rows_write(*self.states, states, at, group=64)
        slot = (torch.arange(n, device="cuda") + at) % CAPACITY
        self.begins[slot] = begins
        for to, v in zip((self.tidx, self.tlogit, self.tlse), top):
            to[slot] = v
        self.tree.add(n)
        self.begins[self.tree.cursor] = True  # what lies behind the newest row does not follow it


def slots_ahead(idx, ahead, cursor):
    """The slots `ahead` of idx; -1, which is no slot, where the newest row comes
    before them: what lies there is of an older episode, or not yet written."""
    newer = (cursor - 1 - idx) % CAPACITY
    return torch.where(ahead <= newer, (idx + ahead) % CAPACITY, -1)


class Student:
    """rows -> (values, gates) -> gated linear recurrence -> logits."""

    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(0)
        self.w = [torch.randn(DIM, 2 * HIDDEN, device="cuda", generator=g) / DIM ** 0.5,
                  torch.randn(HIDDEN, VOCAB, device="cuda", generator=g) / HIDDEN ** 0.5]
        self.m = [torch.zeros_like(w) for w in self.w]
        self.v = [torch.zeros_like(w) for w in self.w]
        self.t = 0

    def step(self, rows, state, begins):
        """One token for each actor; state is updated in place."""
        p = rows @ self.w[0]
        per.per_scan_step(p[:, :HIDDEN], p[:, HIDDEN:], state, reset=begins)

    def learn(self, replay, lr=3e-3):
        u = torch.rand(BATCH, device="cuda")
        s = replay.tree.sample(u, beta=0.4)
        idx, w = s["idx"], s["w"]
        rows = per.per_rows_read(*replay.rows, idx, window=WINDOW, group=0)
        h0 = per.per_rows_read(*replay.states, idx, group=64)[:, 0].contiguous()
        slot = (idx[:, None] + torch.arange(WINDOW, device="cuda")) % CAPACITY
        begins = replay.begins[slot]

        p = rows @ self.w[0]
        x, g = p[..., :HIDDEN], p[..., HIDDEN:]
        y, _, carries = per.per_scan_forward(x, g, reset=begins, h0=h0)
        flat = y.view(-1, HIDDEN)
        logits = flat @ self.w[1]
        flat_slot = slot.view(-1)
        loss, dlogits = per.per_distill(
            logits, replay.tidx[flat_slot], replay.tlogit[flat_slot], tlse=replay.tlse[flat_slot],
            temperature=TEMPERATURE, weight=(w / (BATCH * WINDOW)).repeat_interleave(WINDOW), grad=logits)

        dw1 = flat.t() @ dlogits
        dy = (dlogits @ self.w[1].t()).view_as(y)
        dp = torch.empty_like(p)
        per.per_scan_backward(x, g, carries, dy, reset=begins, dx=dp[..., :HIDDEN], dg=dp[..., HIDDEN:])
        dw0 = rows.view(-1, DIM).t() @ dp.view(-1, 2 * HIDDEN)

        self.t += 1
        for w_, m, v, d in zip(self.w, self.m, self.v, (dw0, dw1)):  # Adam
            m.mul_(0.9).add_(d, alpha=0.1)
            v.mul_(0.99).addcmul_(d, d, value=0.01)
            w_.sub_(lr * (m / (1 - 0.9 ** self.t)) / ((v / (1 - 0.99 ** self.t)).sqrt() + 1e-8))

        seq = loss.view(BATCH, WINDOW)
        replay.tree.update(idx, (0.9 * seq.amax(1) + 0.1 * seq.mean(1)).contiguous())
        # the state before the slot half a window on, with the weights that made it
        half = WINDOW // 2
        per.per_rows_write_at(*replay.states, y[:, half - 1], slots_ahead(idx, half, replay.tree.cursor),
                              replay.claims, group=64)
        return loss.mean()


class Teacher:
    """A fixed recurrence of its own, whose top logits and normaliser are kept."""

    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(1)
        self.a = torch.randn(DIM, HIDDEN, device="cuda", generator=g) / DIM ** 0.5
        self.b = torch.randn(HIDDEN, VOCAB, device="cuda", generator=g) * 3 / HIDDEN ** 0.5

    def __call__(self, rows, begins):
        gate = torch.full((1, rows.shape[0], HIDDEN), 1.5, device="cuda")
        y, _, _ = per.per_scan_forward((rows @ self.a)[None], gate, reset=begins[None])
        z = y[0] @ self.b
        t, i = z.topk(K, 1)
        return i.to(torch.int32), t, torch.logsumexp(z / TEMPERATURE, 1)


def collect(student, teacher, replay, n, gen):
    """ACTORS episodes of n rows, the student's states stepped beside them."""
    rows = torch.randn(ACTORS, n, DIM, device="cuda", generator=gen)
    state = torch.zeros(ACTORS, HIDDEN, device="cuda")
    states = torch.empty(ACTORS, n, HIDDEN, device="cuda")
    begins = torch.zeros(ACTORS, n, dtype=torch.bool, device="cuda")
    begins[:, 0] = True
    for t in range(n):
        states[:, t] = state
        student.step(rows[:, t], state, begins[:, t].contiguous())
    for a in range(ACTORS):
        replay.add(rows[a], states[a], begins[a], teacher(rows[a], begins[a]))


def main(steps=200, say=print):
    gen = torch.Generator(device="cuda").manual_seed(2)
    torch.manual_seed(3)
    replay, student, teacher = Replay(), Student(), Teacher()
    collect(student, teacher, replay, 100, gen)
    losses = []
    for k in range(steps):
        if k and k % 50 == 0:
            collect(student, teacher, replay, 20, gen)
        losses.append(student.learn(replay))
        if say and (k % 20 == 0 or k == steps - 1):
            say("step %4d  mean loss of the sampled rows %.4f  filled %d" % (k, float(losses[-1]), replay.tree.size))
    out = torch.stack(losses).cpu()
    replay.tree.close()
    return out


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=200)
    main(ap.parse_args().steps)
